"""Argument checks of the calls around the layer (moe_add_rmsnorm, moe_route_scores, moe_swiglu_i8,
moe_matmul_i8): made on the host before anything is enqueued, so no GPU is needed. Pointers are
fakes that no call below gets to use."""
import ctypes
import os

import pytest
import torch

from moe_routed_expert_route_amd import binding as B

ARG, SHAPE, OK = -1, -3, 0
P, P2, P3, P4, P5 = (i << 32 for i in range(1, 6))   # far from each other
NAN, INF = float("nan"), float("inf")

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

NORM = dict(dtype=1, x=P, ldx=64, res=P2, ldres=64, w_dtype=1, weight=P3, eps=1e-6, rows=4, n=64, res_out=P2, ldro=64,
            y_dtype=1, y=P4, ldy=64, q=P5, ldq=64, scale=P5 + 4096, q8_1=None)
ROUTE = dict(dtype=1, logits=P, ld=64, T=4, E=64, k=8, score=1, bias=P2, n_groups=8, keep=4, top=2, renorm=1, factor=1.0,
             ids=P3, w=P4)
SWIGLU = dict(dtype=2, g=P, ldg=128, u=P + 128, ldu=128, rows=4, n=64, q=P3, ldq=64, scale=P4)
MATMUL = dict(a=P, lda=64, sa=P2, b=P3, ldb=64, sb=P4, M=4, N=32, K=64, c_dtype=2, c=P5, ldc=32, accumulate=0)
CALLS = {"moe_add_rmsnorm": NORM, "moe_route_scores": ROUTE, "moe_swiglu_i8": SWIGLU, "moe_matmul_i8": MATMUL}

BAD = [
    ("moe_add_rmsnorm", dict(dtype=0), ARG), ("moe_add_rmsnorm", dict(dtype=4), ARG), ("moe_add_rmsnorm", dict(w_dtype=9), ARG),
    ("moe_add_rmsnorm", dict(y_dtype=0), ARG), ("moe_add_rmsnorm", dict(rows=-1), ARG), ("moe_add_rmsnorm", dict(n=0), SHAPE),
    ("moe_add_rmsnorm", dict(n=16385, ldx=20000, ldres=20000, ldro=20000, ldy=20000, ldq=20000), SHAPE),
    ("moe_add_rmsnorm", dict(eps=0.0), ARG), ("moe_add_rmsnorm", dict(eps=-1.0), ARG), ("moe_add_rmsnorm", dict(eps=NAN), ARG),
    ("moe_add_rmsnorm", dict(eps=INF), ARG), ("moe_add_rmsnorm", dict(x=None), ARG), ("moe_add_rmsnorm", dict(weight=None), ARG),
    ("moe_add_rmsnorm", dict(q=None), ARG), ("moe_add_rmsnorm", dict(scale=None), ARG),
    ("moe_add_rmsnorm", dict(res_out=None, y=None, q=None, scale=None), ARG),
    ("moe_add_rmsnorm", dict(ldx=63), ARG), ("moe_add_rmsnorm", dict(ldres=63), ARG), ("moe_add_rmsnorm", dict(ldro=63), ARG),
    ("moe_add_rmsnorm", dict(ldy=63), ARG), ("moe_add_rmsnorm", dict(ldq=63), ARG), ("moe_add_rmsnorm", dict(x=P + 2), ARG),
    ("moe_add_rmsnorm", dict(y=P4 + 1), ARG), ("moe_add_rmsnorm", dict(scale=P5 + 4098), ARG),
    ("moe_add_rmsnorm", dict(n=63, q8_1=P4 + (1 << 20)), SHAPE), ("moe_add_rmsnorm", dict(q8_1=P4 + 2 + (1 << 20)), ARG),
    ("moe_add_rmsnorm", dict(res_out=P2 + 4), ARG), ("moe_add_rmsnorm", dict(res_out=P2, ldro=65), ARG),
    ("moe_add_rmsnorm", dict(y=P), ARG), ("moe_add_rmsnorm", dict(q=P + 100), ARG), ("moe_add_rmsnorm", dict(q8_1=P2 + 64), ARG),
    ("moe_add_rmsnorm", dict(q=P4 + 64), ARG), ("moe_add_rmsnorm", dict(scale=P5 + 16), ARG), ("moe_add_rmsnorm", dict(y=P3), ARG),
    ("moe_add_rmsnorm", dict(rows=1 << 22), SHAPE), ("moe_add_rmsnorm", dict(y=P2 + 128, ldy=32), ARG),
    ("moe_add_rmsnorm", dict(x=P, ldx=128, y=P + 192, ldy=128), ARG), ("moe_add_rmsnorm", dict(x=P, ldx=128, y=P - 192, ldy=128), ARG),
    ("moe_route_scores", dict(T=1 << 22), SHAPE), ("moe_route_scores", dict(ids=P + 64), ARG), ("moe_route_scores", dict(w=P3 + 64), ARG),
    ("moe_swiglu_i8", dict(rows=1 << 22), SHAPE), ("moe_swiglu_i8", dict(scale=P3 + 8), ARG),
    ("moe_matmul_i8", dict(N=2147483137, ldc=1 << 31), SHAPE), ("moe_matmul_i8", dict(M=2147483137), SHAPE),
    ("moe_matmul_i8", dict(a=1 << 50, b=1 << 51, sa=1 << 52, sb=1 << 53, c=1 << 54, N=1 << 28, ldc=1 << 28), SHAPE),
    ("moe_matmul_i8", dict(c=P + 64), ARG), ("moe_matmul_i8", dict(c=P3 + 32), ARG), ("moe_matmul_i8", dict(c=P2 - 8), ARG),
    ("moe_matmul_i8", dict(c=P4 + 64), ARG), ("moe_route_scores", dict(dtype=0), ARG), ("moe_route_scores", dict(T=-1), ARG), ("moe_route_scores", dict(E=0, ld=64), ARG),
    ("moe_route_scores", dict(E=1025, ld=2048, n_groups=1, keep=1), ARG), ("moe_route_scores", dict(k=0), ARG),
    ("moe_route_scores", dict(k=33), ARG), ("moe_route_scores", dict(k=9, keep=1), ARG), ("moe_route_scores", dict(score=0), ARG),
    ("moe_route_scores", dict(score=3), ARG), ("moe_route_scores", dict(n_groups=0), ARG), ("moe_route_scores", dict(n_groups=7), ARG),
    ("moe_route_scores", dict(E=650, ld=650, n_groups=65, keep=65), ARG), ("moe_route_scores", dict(keep=0), ARG),
    ("moe_route_scores", dict(keep=9), ARG), ("moe_route_scores", dict(top=0), ARG), ("moe_route_scores", dict(top=3), ARG),
    ("moe_route_scores", dict(E=8, ld=8, n_groups=8, keep=8, k=2, top=2), ARG), ("moe_route_scores", dict(renorm=2), ARG),
    ("moe_route_scores", dict(factor=NAN), ARG), ("moe_route_scores", dict(ld=63), ARG), ("moe_route_scores", dict(logits=None), ARG),
    ("moe_route_scores", dict(ids=None), ARG), ("moe_route_scores", dict(w=None), ARG), ("moe_route_scores", dict(logits=P + 2), ARG),
    ("moe_route_scores", dict(ids=P3 + 2), ARG), ("moe_route_scores", dict(bias=P2 + 1), ARG),
    ("moe_swiglu_i8", dict(dtype=7), ARG), ("moe_swiglu_i8", dict(rows=-1), ARG), ("moe_swiglu_i8", dict(n=0), SHAPE),
    ("moe_swiglu_i8", dict(n=16385, ldg=40000, ldu=40000, ldq=20000), SHAPE), ("moe_swiglu_i8", dict(g=None), ARG),
    ("moe_swiglu_i8", dict(u=None), ARG), ("moe_swiglu_i8", dict(q=None), ARG), ("moe_swiglu_i8", dict(scale=None), ARG),
    ("moe_swiglu_i8", dict(ldg=63), ARG), ("moe_swiglu_i8", dict(ldu=63), ARG), ("moe_swiglu_i8", dict(ldq=63), ARG),
    ("moe_swiglu_i8", dict(g=P + 1), ARG), ("moe_swiglu_i8", dict(u=P + 129), ARG), ("moe_swiglu_i8", dict(q=P + 64), ARG),
    ("moe_matmul_i8", dict(c_dtype=0), ARG), ("moe_matmul_i8", dict(M=-1), ARG), ("moe_matmul_i8", dict(N=-1), ARG),
    ("moe_matmul_i8", dict(K=0), SHAPE), ("moe_matmul_i8", dict(K=131072, lda=1 << 20, ldb=1 << 20), SHAPE),
    ("moe_matmul_i8", dict(a=None), ARG), ("moe_matmul_i8", dict(b=None), ARG), ("moe_matmul_i8", dict(sa=None), ARG),
    ("moe_matmul_i8", dict(sb=None), ARG), ("moe_matmul_i8", dict(c=None), ARG), ("moe_matmul_i8", dict(lda=63), ARG),
    ("moe_matmul_i8", dict(ldb=63), ARG), ("moe_matmul_i8", dict(ldc=31), ARG), ("moe_matmul_i8", dict(sa=P2 + 2), ARG),
    ("moe_matmul_i8", dict(c=P5 + 1), ARG), ("moe_matmul_i8", dict(accumulate=2), ARG),
    # calls of no rows succeed without their row pointers, once their scalars are sound
    ("moe_add_rmsnorm", dict(rows=0, x=None, res=None, y=None, q=None, scale=None), OK),
    ("moe_route_scores", dict(T=0, logits=None, ids=None, w=None), OK),
    ("moe_swiglu_i8", dict(rows=0, g=None, u=None, q=None, scale=None), OK),
    ("moe_matmul_i8", dict(M=0, a=None, sa=None, c=None), OK), ("moe_matmul_i8", dict(N=0, b=None, sb=None, c=None), OK),
]


@pytest.mark.parametrize("name,change,want", BAD, ids=[f"{n}-{','.join(f'{k}={v}' for k, v in c.items())}" for n, c, _ in BAD])
def test_refused_on_the_host(name, change, want):
    args = dict(CALLS[name])
    assert set(change) <= set(args)
    args.update(change)
    assert getattr(B.lib(), name)(None, *args.values()) == want


def test_binding_refuses_tensors_of_the_cpu():
    x, q = torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.int8)
    s = torch.zeros(2)
    for call in (lambda: B.moe_add_rmsnorm(x, torch.ones(64), 1e-6, y=x), lambda: B.moe_route_scores(x, 2),
                 lambda: B.moe_swiglu_i8(x, x, q, s), lambda: B.moe_matmul_i8(q, s, q, s)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_binding_refuses_shapes_types_and_strides():
    x = torch.zeros(2, 64)   # the checks themselves, with the CPU's index (-1) as the call's device
    for want, t, shape, dtypes, device in (("shape", x, (2, 63), (torch.float32,), -1), ("rows", x[0], None, (torch.float32,), -1),
                                           ("int8", x, None, (torch.int8,), -1), ("call's GPU", x, None, (torch.float32,), 0),
                                           ("next to each other", x.t(), None, (torch.float32,), -1)):
        with pytest.raises(ValueError, match=want):
            B._rows("call", "t", t, shape, dtypes, device)
    assert B._rows("call", "t", torch.zeros(3, 90)[:, 5:69], (3, 64), (torch.float32,), -1) == 90
    assert B._rows("call", "t", torch.zeros(1, 64), None, (torch.float32,), -1) == 64
    for t in (torch.zeros(8)[::2], torch.zeros(5), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 1)):
        with pytest.raises(ValueError, match="not contiguous"):
            B._packed("call", "t", t, (4,), torch.float32, -1)
    with pytest.raises(ValueError, match="call's GPU"):
        B._packed("call", "t", torch.zeros(4), (4,), torch.float32, 0)


@pytest.mark.parametrize("name,change", [
    ("moe_add_rmsnorm", dict(rows=1, res_out=P3)),                       # the weight's row is not the residual's
    ("moe_route_scores", dict(ids=P2)), ("moe_route_scores", dict(w=P2 + 128)),   # over the bias
])
def test_refuses_outputs_over_the_weight_and_the_bias(name, change):
    assert getattr(B.lib(), name)(None, *dict(CALLS[name], **change).values()) == ARG


def test_binding_refuses_sizes_past_32_bits():
    for shape in ((1 << 31, 1), (1, (1 << 32) + 16)):   # of no memory: one element, expanded
        with pytest.raises(ValueError, match="past 32 bits"):
            B._rows("call", "t", torch.zeros(1, 1).expand(shape), None, (torch.float32,), -1)


HIP = -4


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch kernels on pointers that are fakes")
@pytest.mark.parametrize("M,N,K,launches", [
    (16, 134217712, 64, True), (16, 134217713, 64, False),     # 512 threads for 16 channels
    (17, 134217712, 64, True), (17, 134217713, 64, True), (32, 1 << 28, 1024, True), (17, 1 << 27, 1025, True),
    (33, (1 << 30) - 64, 16, True), (33, 1 << 30, 16, True),   # 64 x 64 tiles up to 2^30 - 64 channels, then larger ones
    (257, 1 << 29, 16, True), (1 << 30, 33, 16, True), (256, 2147483136, 16, True), (2147483136, 17, 16, True),
    (1 << 19, (1 << 20) - 256, 16, True), (1 << 19, (1 << 20) - 255, 16, False), (2147483136, 257, 16, False)])
def test_matmul_sizes_are_refused_only_past_a_launch(M, N, K, launches):
    """Without a GPU a call that passes its checks ends in the launch's own error."""
    far = dict(a=1 << 50, b=1 << 52, sa=1 << 54, sb=1 << 55, c=1 << 57)
    got = getattr(B.lib(), "moe_matmul_i8")(None, *dict(MATMUL, **far, M=M, N=N, K=K, lda=1024 + K, ldb=1024 + K, ldc=N).values())
    assert got == (HIP if launches else SHAPE)


FAR = {"moe_add_rmsnorm": dict(scale=P5 + (1 << 31)), "moe_route_scores": {}, "moe_swiglu_i8": {}, "moe_matmul_i8": dict(ldc=1 << 20)}
STRIDES = [("moe_add_rmsnorm", "rows", ("ldx", "ldres", "ldro", "ldy", "ldq")), ("moe_route_scores", "T", ("ld",)),
           ("moe_swiglu_i8", "rows", ("ldg", "ldu", "ldq")), ("moe_matmul_i8", "M", ("lda", "ldc")), ("moe_matmul_i8", "N", ("ldb",))]


@pytest.mark.parametrize("rows", [1, 2, 5, 1 << 20])
@pytest.mark.parametrize("ld", [(1 << 50) + 1, 1 << 60, 1 << 62, (1 << 62) + 1, (1 << 63) - 1])
@pytest.mark.parametrize("name,count,strides", STRIDES)
def test_strides_past_any_memory_are_refused(name, count, strides, ld, rows):
    """Each stride alone and all together: in bytes, or times the rows, they wrap in 64 bits."""
    for change in [{s: ld} for s in strides] + [{s: ld for s in strides}, {s: (1 << 50) // rows + 1 for s in strides}]:
        args = dict(CALLS[name], **{**FAR[name], count: rows, **change})
        assert getattr(B.lib(), name)(None, *args.values()) == ARG, change


def test_huge_strides_of_overlapping_rows_are_refused():
    for rows, ld in ((1, 1 << 62), (5, 1 << 60), (3, 1 << 61), (1 << 20, 1 << 42)):
        args = dict(NORM, rows=rows, res=None, res_out=None, q=None, scale=None, ldx=ld, ldy=ld, y=P + 16)
        assert B.lib().moe_add_rmsnorm(None, *args.values()) == ARG


@pytest.mark.parametrize("q,want", [(P + 16, ARG), (P + 255, ARG), (P - 63, ARG), (P + 256, HIP), (P - 64, HIP), (P + (1 << 20), HIP)])
@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch kernels on pointers that are fakes")
def test_one_row_of_any_stride_overlaps_by_its_bytes(q, want):
    args = dict(NORM, rows=1, res=None, res_out=None, y=None, q=q, scale=P4, ldx=1 << 50, ldq=1 << 48)
    assert B.lib().moe_add_rmsnorm(None, *args.values()) == want


@pytest.mark.parametrize("factor", [INF, -INF])
def test_route_factor_has_to_be_finite(factor):
    """A masked token's weights are 0, which no infinite factor leaves."""
    assert B.lib().moe_route_scores(None, *dict(ROUTE, factor=factor).values()) == ARG


@pytest.mark.parametrize("c,want", [(P3 + 64, HIP), (P3 + 192, HIP), (P3 + 62, ARG), (P3 + 194, ARG), (P3 + 256, ARG), (P3 + 31 * 256 + 64, HIP),
                                    (P3 - 64, HIP), (P3 - 62, ARG)])
@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch kernels on pointers that are fakes")
def test_one_row_of_results_between_the_rows_of_an_input(c, want):
    """Rows of 64 bytes, 256 apart, and one row of C of 64 bytes, whatever its stride."""
    for ldc in (32, 128, 1000):
        assert B.lib().moe_matmul_i8(None, *dict(MATMUL, M=1, ldb=256, c=c, ldc=ldc).values()) == want
    args = dict(NORM, rows=1, res=None, res_out=P, ldro=100, y=None, q=None, scale=None)   # in place, its one row
    assert B.lib().moe_add_rmsnorm(None, *args.values()) == HIP
