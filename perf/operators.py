"""The operators around a routed-expert layer, as workloads to be timed and checked: the norm before it
(residual added, output in 8 bits), the router, and the shared expert's 8-bit matrix product and SwiGLU.

``own`` false: the operators in plain torch operations. ``own`` true: the library's entry points.
"""
import numpy as np
import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the token of a decode step at the library's headline width: the decode path takes float rows,
        # the shared expert int8 rows
        dict(name="norm 1x2560 f32", op="norm", rows=1, n=2560, type="f32", y=True, i8=True, q8_1=False),
        # a 512-token prompt in front of the prompt path (q8_1 rows), the router (float rows) and the
        # shared expert (int8 rows)
        dict(name="norm 512x2560 f32 all", op="norm", rows=512, n=2560, type="f32", y=True, i8=True, q8_1=True),
        # a long prompt's residual stream in bfloat16 in front of an 8-bit product
        dict(name="norm 8192x4096 bf16", op="norm", rows=8192, n=4096, type="bf16", y=False, i8=True, q8_1=False),
        # the headline layer's router for one token: softmax, 8 of 128
        dict(name="route 1x128 softmax", op="route", T=1, E=128, k=8, type="f32", score="softmax", bias=False,
             groups=1, keep=1, top=1, renorm=True, masked=False),
        # a prompt through a router with sigmoid scores, a balance bias and limited groups
        dict(name="route 512x256 groups", op="route", T=512, E=256, k=8, type="f32", score="sigmoid", bias=True,
             groups=8, keep=4, top=2, renorm=True, masked=False),
        # a batch of long prompts, bfloat16 logits (equal ones among them), some experts and rows masked
        dict(name="route 16384x256 bf16 masked", op="route", T=16384, E=256, k=8, type="bf16", score="softmax",
             bias=False, groups=1, keep=1, top=1, renorm=True, masked=True),
        # the shared expert's gate and up product for one token, both matrices stacked
        dict(name="matmul 1x1536x2560", op="matmul", M=1, N=1536, K=2560, out="f32"),
        # a batch of decode streams
        dict(name="matmul 64x5120x2560", op="matmul", M=64, N=5120, K=2560, out="bf16"),
        # a ragged prompt, odd in every size
        dict(name="matmul 509x2561x1283", op="matmul", M=509, N=2561, K=1283, out="f32"),
        # long prompts through a wide dense layer
        dict(name="matmul 8192x8192x4096", op="matmul", M=8192, N=8192, K=4096, out="bf16"),
        # the shared expert's activation for a window of four tokens
        dict(name="swiglu 4x768 f32", op="swiglu", rows=4, n=768, type="f32"),
        # and for long prompts at an odd width
        dict(name="swiglu 4096x5461 bf16", op="swiglu", rows=4096, n=5461, type="bf16"),
    ]


def _size(rng, lo, hi):
    """A size of lo..hi, even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def _width(rng, lo, hi):
    """A row length: half of them multiples of 64, the others as they come, odd ones among them."""
    n = _size(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm", "route", "matmul", "swiglu"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        n = _width(rng, 33, 8192)
        rows = _size(rng, 1, min(8192, (1 << 23) // n))
        return dict(op=op, rows=rows, n=n, type=kind, y=rng.random() < 0.5, i8=True,
                    q8_1=n % 32 == 0 and rng.random() < 0.5)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _size(rng, 4, 512 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(12, keep * (E // groups)))
        return dict(op=op, T=_size(rng, 1, min(16384, (1 << 21) // E)), E=E, k=k, type=kind, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.7, masked=rng.random() < 0.3)
    if op == "matmul":
        return dict(op=op, M=_size(rng, 1, 4096), N=_width(rng, 64, 8192), K=_width(rng, 64, 8192), out=kind)
    n = _width(rng, 33, 8192)
    return dict(op=op, rows=_size(rng, 1, min(8192, (1 << 23) // n)), n=n, type=kind)


def work(case):
    op = case["op"]
    if op == "norm":
        e, s = case["rows"] * case["n"], SIZE[case["type"]]
        # x, the residual and its sum; the float rows; int8 rows with scales; 36-byte blocks of 32
        b = e * 3 * s + case["n"] * s + (4 * e if case["y"] else 0)
        b += (e + 4 * case["rows"] if case["i8"] else 0) + (e // 32 * 36 if case["q8_1"] else 0)
        return {"bytes": b, "flops": 10 * e}
    if op == "route":
        e = case["T"] * case["E"]
        return {"bytes": e * SIZE[case["type"]] + case["T"] * case["k"] * 8 + (4 * case["E"] if case["bias"] else 0),
                "flops": 10 * e}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    e = case["rows"] * case["n"]
    return {"bytes": e * (2 * SIZE[case["type"]] + 1) + 4 * case["rows"], "flops": 10 * e}


# ------------------------------------------------------------------ inputs ---------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    st, op = {"case": case}, case["op"]
    if op == "norm":
        rows, n, t = case["rows"], case["n"], DTYPES[case["type"]]
        # a residual stream: a few channels far larger than the others, tokens of different size
        channel = torch.exp(0.5 * randn(n)) * torch.where(randn(n) > 2.5, 8.0, 1.0)
        st["res"] = (randn(rows, n) * channel * torch.exp(0.3 * randn(rows, 1))).to(t)
        st["x"] = (0.3 * randn(rows, n)).to(t)
        st["weight"] = (1.0 + 0.2 * randn(n)).to(t)
        st["sum"] = torch.empty_like(st["x"])
    elif op == "route":
        T, E = case["T"], case["E"]
        logits = 2.0 * randn(T, E)
        if case["masked"]:   # about an eighth of the experts, and every expert of a few padded tokens
            logits = logits.masked_fill(randn(T, E) > 1.15, float("-inf"))
            logits = logits.masked_fill(randn(T, 1) > 1.9, float("-inf"))
        st["logits"] = logits.to(DTYPES[case["type"]])
        st["bias"] = 0.1 * randn(E) if case["bias"] else None
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        st["a"] = torch.round(30.0 * randn(M, K)).clamp_(-127, 127).to(torch.int8)
        st["b"] = torch.round(36.0 * randn(N, K)).clamp_(-127, 127).to(torch.int8)
        st["sa"] = 0.03 * torch.exp(0.3 * randn(M))
        st["sb"] = 0.0005 * torch.exp(0.3 * randn(N))
    else:
        rows, n, t = case["rows"], case["n"], DTYPES[case["type"]]
        # the two halves of one product's rows: gate columns, then up columns
        st["gu"] = (1.5 * randn(rows, 2 * n) * torch.exp(0.3 * randn(rows, 1))).to(t)
    return st


# ------------------------------------------------------------------ plain forms ----------------

def _codes(y, d):
    """q8_1's codes of float32 values y in blocks (last axis) of scale d: the float32 quotient rounded
    to the nearest integer, halves away from zero."""
    v = (y / torch.where(d > 0, d, torch.ones_like(d))).double()
    return torch.sign(v) * torch.floor(v.abs() + 0.5).clamp_(max=127.0)


def _scale(y):
    d = y.abs().amax(-1, keepdim=True)
    return d / torch.full_like(d, 127.0)   # by a number, torch multiplies by its rounded reciprocal


def _int8_rows(y):
    d = _scale(y)
    return _codes(y, d).float() * d


def _plain_norm(st):
    case, x, res = st["case"], st["x"], st["res"]
    r = (x.float() + res.float()).to(x.dtype)
    r64 = r.double()
    # 64 bits: a value next to a code's border has to fall on its own side of it
    y = (r64 * torch.rsqrt((r64 * r64).mean(-1, keepdim=True) + EPS) * st["weight"].double()).float()
    out = {"sum": r}
    if case["y"]:
        out["y"] = y
    if case["i8"]:
        out["i8"] = _int8_rows(y)
    if case["q8_1"]:
        blocks = y.view(y.shape[0], -1, 32)
        d = _scale(blocks)
        q = _codes(blocks, d).float()
        d16 = d.half()
        out["q8_1"] = (q * d16.float()).view_as(y)
        out["block sums"] = (d16.float() * q.sum(-1, keepdim=True)).half().squeeze(-1)
    return out


def _plain_route(st):
    case = st["case"]
    # 64 bits: two experts next to each other keep the order that they have
    logits = st["logits"].double()
    masked = torch.isneginf(logits) | torch.isnan(logits)
    logits = logits.masked_fill(masked, float("-inf"))
    if case["score"] == "softmax":
        top = logits.amax(-1, keepdim=True)
        e = torch.exp(logits - top.masked_fill(torch.isneginf(top), 0.0))
        total = e.sum(-1, keepdim=True)
        s = e / total.masked_fill(total == 0, 1.0)
    else:
        s = 1.0 / (1.0 + torch.exp(-logits))
    c = s + st["bias"].double() if case["bias"] else s
    c = c.masked_fill(masked, float("-inf"))
    if case["groups"] > 1:
        T, E, G = case["T"], case["E"], case["groups"]
        best = torch.sort(c.view(T, G, E // G), dim=-1, descending=True).values[..., :case["top"]]
        score = torch.where(torch.isneginf(best), torch.zeros_like(best), best).sum(-1)
        score = score.masked_fill(torch.isneginf(best[..., 0]), float("-inf"))
        kept = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :case["keep"]]
        out = torch.ones(T, G, dtype=torch.bool, device=c.device).scatter_(1, kept, False)
        # experts of the other groups come after the masked ones of these
        c = c.clamp(min=-1e30).masked_fill(out.repeat_interleave(E // G, 1), float("-inf"))
    ids = torch.sort(c, dim=-1, descending=True, stable=True).indices[:, :case["k"]]
    w = torch.gather(s, 1, ids)
    if case["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / total.masked_fill(total == 0, 1.0)
    return {"ids": ids.int(), "w": w.float()}


def _plain_matmul(st):
    sums = st["a"].float() @ st["b"].float().t()
    return {"c": (sums * st["sa"][:, None] * st["sb"]).to(DTYPES[st["case"]["out"]])}


def _plain_swiglu(st):
    n = st["case"]["n"]
    g, u = st["gu"][:, :n].double(), st["gu"][:, n:].double()   # 64 bits: values next to a code's border
    return {"i8": _int8_rows((g / (1.0 + torch.exp(-g)) * u).float())}


# ------------------------------------------------------------------ the library's calls --------

def _own_norm(st):
    from moe_routed_expert_route_amd import binding as B
    case, x = st["case"], st["x"]
    rows, n = x.shape
    y = torch.empty((rows, n), dtype=torch.float32, device=x.device) if case["y"] else None
    q, d = B.i8_rows(rows, n, x.device) if case["i8"] else (None, None)
    blocks = torch.empty((rows, n // 32 * 36), dtype=torch.uint8, device=x.device) if case["q8_1"] else None
    B.moe_add_rmsnorm(x, st["weight"], EPS, res=st["res"], res_out=st["sum"], y=y, q=q, scale=d, q8_1=blocks)
    out = {"sum": st["sum"]}
    if case["y"]:
        out["y"] = y
    if case["i8"]:
        out["i8"] = torch.mul(q, d[:, None])
    if case["q8_1"]:
        blocks = blocks.view(rows, n // 32, 36)
        head = blocks[..., :4].contiguous().view(torch.float16)
        out["q8_1"] = torch.mul(blocks[..., 4:].view(torch.int8), head[..., :1].float()).view(rows, n)
        out["block sums"] = head[..., 1].contiguous()
    return out


def _own_route(st):
    from moe_routed_expert_route_amd import binding as B
    case = st["case"]
    score = B.SCORE_SOFTMAX if case["score"] == "softmax" else B.SCORE_SIGMOID
    ids, w = B.moe_route_scores(st["logits"], case["k"], score=score, bias=st["bias"], n_groups=case["groups"],
                                keep_groups=case["keep"], group_top=case["top"], renorm=case["renorm"])
    return {"ids": ids, "w": w}


def _own_matmul(st):
    from moe_routed_expert_route_amd import binding as B
    return {"c": B.moe_matmul_i8(st["a"], st["sa"], st["b"], st["sb"], dtype=DTYPES[st["case"]["out"]])}


def _own_swiglu(st):
    from moe_routed_expert_route_amd import binding as B
    n = st["case"]["n"]
    q, d = B.moe_swiglu_i8(st["gu"][:, :n], st["gu"][:, n:])
    return {"i8": torch.mul(q, d[:, None])}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "route": _own_route, "matmul": _own_matmul, "swiglu": _own_swiglu}[op](state)
    return {"norm": _plain_norm, "route": _plain_route, "matmul": _plain_matmul, "swiglu": _plain_swiglu}[op](state)


# ------------------------------------------------------------------ in 64 bits -----------------

def _quantized(y32, axis):
    """The values that 8-bit codes of float32 rows stand for, as (codes, float32 scale) in float64. The
    definition's own roundings (the scale and the quotient in float32) are part of it."""
    d = (np.abs(y32).max(axis, keepdims=True) / np.float32(127)).astype(np.float32)
    v = np.divide(y32, d, out=np.zeros_like(y32), where=d > 0).astype(np.float64)
    t = np.trunc(v)
    return np.clip(t + np.where(np.abs(v - t) >= 0.5, np.sign(v), 0.0), -127, 127), d.astype(np.float64)


def _host(t):
    return t.detach().cpu().double().numpy()


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "matmul":
        c = torch.matmul(st["a"].double(), st["b"].double().t())   # whole numbers below 2^53
        return {"c": c * torch.outer(st["sa"].double(), st["sb"].double())}
    if op == "norm":
        total = _host(st["x"]) + _host(st["res"])
        r = _host(torch.from_numpy(total).to(DTYPES[case["type"]]))
        mean_square = np.einsum("ij,ij->i", r, r) / case["n"]
        y = r / np.sqrt(mean_square + EPS)[:, None] * _host(st["weight"])[None]
        out = {"sum": total}
        if case["y"]:
            out["y"] = y
        y32 = y.astype(np.float32)
        if case["i8"]:
            q, d = _quantized(y32, 1)
            out["i8"] = q * d
        if case["q8_1"]:
            q, d = _quantized(y32.reshape(case["rows"], -1, 32), 2)
            d = d.astype(np.float16).astype(np.float64)   # the block keeps its scale in 16 bits
            out["q8_1"] = (q * d).reshape(y.shape)
            out["block sums"] = q.sum(2) * d[..., 0]
        return out
    if op == "swiglu":
        gu = _host(st["gu"])
        g, u = gu[:, :case["n"]], gu[:, case["n"]:]
        q, d = _quantized((u * g / (np.exp(-g) + 1.0)).astype(np.float32), 1)
        return {"i8": q * d}
    return _exact_route(case, _host(st["logits"]), None if st["bias"] is None else _host(st["bias"]))


def _exact_route(case, logits, bias):
    T, E, G = case["T"], case["E"], case["groups"]
    live = np.isfinite(logits)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        if case["score"] == "softmax":
            peak = np.where(live, logits, -np.inf).max(1, keepdims=True)
            s = np.where(live, np.exp(np.where(live, logits - peak, 0.0)), 0.0)
            s = np.nan_to_num(s / s.sum(1, keepdims=True))
        else:
            s = np.where(live, 1.0 / (1.0 + np.exp(-logits)), 0.0)
    c = s if bias is None else s + bias[None]
    # three classes, one after the other: live experts of kept groups, masked ones of them, the rest
    kept = np.ones((T, E), dtype=bool)
    if G > 1:
        per = np.where(live, c, -np.inf).reshape(T, G, E // G)
        best = -np.sort(-per, axis=2)[:, :, :case["top"]]
        score = np.where(np.isfinite(best[:, :, 0]), np.where(np.isfinite(best), best, 0.0).sum(2), -np.inf)
        order = np.argsort(-score, axis=1, kind="stable")[:, :case["keep"]]
        kept = np.zeros((T, G), dtype=bool)
        np.put_along_axis(kept, order, True, 1)
        kept = np.repeat(kept, E // G, axis=1)
    kind = np.where(kept, np.where(live, 0, 1), 2)
    index = np.broadcast_to(np.arange(E), (T, E))
    ids = np.lexsort((index, np.where(live, -c, 0.0), kind), axis=1)[:, :case["k"]]
    w = np.take_along_axis(s, ids, 1)
    if case["renorm"]:
        total = w.sum(1, keepdims=True)
        w = w / np.where(total == 0, 1.0, total)
    return {"ids": ids.astype(np.int32), "w": w}
