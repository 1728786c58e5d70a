"""The attention half of a decoder layer for windows of drafted tokens, and the scores of its answers, as
workloads to be timed and checked: appending a window's rows to a paged cache (norm of each head, rotation by
position and 8-bit rows on the way), attention of the window's tree over that cache, and log probabilities of
given tokens with entropy and the best alternatives.

``own`` false: the operators in plain torch operations. ``own`` true: the library's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}


def listed():
    return [
        # one token of a decode step behind a prompt of a thousand: 32 heads over 4, normed and rotated
        dict(name="append 1x1 bf16", op="append", seqs=1, T=1, ragged=False, tree=False, pad=0, lo=1000, hi=1000, heads=32, kv=4,
             d=128, rot=128, layout="half", norm=True, amp=1.0, type="bf16", out="bf16", cache="bf16", page=16),
        # 64 decode streams with a tree of four drafted tokens each, the products' float32 rows into 8 bits
        dict(name="append 64x4 f32 i8", op="append", seqs=64, T=4, ragged=False, tree=True, pad=0, lo=16, hi=512, heads=32, kv=8,
             d=128, rot=128, layout="half", norm=True, amp=1.0, type="f32", out="bf16", cache="i8", page=64),
        # ragged prompts, a part of each head rotated as neighbouring pairs, no norm, padded rows behind them
        dict(name="append 5x211 f16 partial", op="append", seqs=5, T=211, ragged=True, tree=False, pad=3, lo=0, hi=700, heads=20,
             kv=5, d=80, rot=36, layout="pairs", norm=False, amp=1.1, type="f16", out="f16", cache="f16", page=16),
        # long prompts in front of an empty cache
        dict(name="append 8x1024 bf16", op="append", seqs=8, T=1024, ragged=False, tree=False, pad=0, lo=0, hi=0, heads=32, kv=8,
             d=128, rot=128, layout="half", norm=True, amp=1.0, type="bf16", out="bf16", cache="bf16", page=256),
        # one token of one stream, where latency counts
        dict(name="attend 1x1 4096 bf16", op="attend", seqs=1, T=1, ragged=False, tree=False, blank=False, pad=0, lo=4095, hi=4095,
             heads=32, kv=4, d=128, type="bf16", cache="bf16", page=16),
        # a tree of four drafted tokens at the end of a long context
        dict(name="attend 1x4 131072 bf16", op="attend", seqs=1, T=4, ragged=False, tree=True, blank=False, pad=0, lo=131000,
             hi=131000, heads=32, kv=4, d=128, type="bf16", cache="bf16", page=256),
        # a batch of streams of different length, windows of four tokens one after the other, a cache in 8 bits
        dict(name="attend 64x4 8192 i8", op="attend", seqs=64, T=4, ragged=False, tree=False, blank=False, pad=0, lo=512, hi=8192,
             heads=32, kv=8, d=128, type="bf16", cache="i8", page=64),
        # the largest trees, where the products count rather than the cache's bytes
        dict(name="attend 8x64 8192 f16", op="attend", seqs=8, T=64, ragged=False, tree=True, blank=False, pad=0, lo=4096, hi=8100,
             heads=64, kv=8, d=128, type="f16", cache="f16", page=32),
        # small ragged trees at an odd head width: empty contexts, a stream without tokens, tokens that see nothing
        dict(name="attend 6x7 1000 ragged", op="attend", seqs=6, T=7, ragged=True, tree=True, blank=True, pad=2, lo=0, hi=1000,
             heads=10, kv=2, d=80, type="bf16", cache="bf16", page=16),
        # the next token of one stream: its probability and five alternatives
        dict(name="logprobs 1x32000 bf16", op="logprobs", rows=1, n=32000, extra=0, given=1, k=5, entropy=True, scale=1.0,
             masked=False, type="bf16"),
        # windows of drafted tokens over an odd vocabulary in padded rows, part of it masked
        dict(name="logprobs 257x50021 f32 masked", op="logprobs", rows=257, n=50021, extra=27, given=4, k=20, entropy=True,
             scale=1.25, masked=True, type="f32"),
        # prompts scored against a wide vocabulary
        dict(name="logprobs 1024x131072 bf16", op="logprobs", rows=1024, n=131072, extra=0, given=1, k=8, entropy=True, scale=1.0,
             masked=False, type="bf16"),
    ]


def _size(rng, lo, hi):
    """A size of lo..hi, even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def _draw(rng):
    op = rng.choice(["append", "attend", "attend", "logprobs"])
    kind = rng.choice(["bf16", "f16"])
    if op == "logprobs":
        n, given = _size(rng, 700, 262144), rng.choice([0, 1, 1, 2, 7])
        return dict(op=op, rows=_size(rng, 1, 1024), n=n, extra=rng.choice([0, 0, -n % 64, 5]), given=given,
                    k=rng.choice([0, 1, 5, 8, 20, 32] if given else [1, 5, 8, 20, 32]), entropy=rng.random() < 0.6,
                    scale=rng.choice([1.0, 1.0, 0.75, 1.5]), masked=rng.random() < 0.3, type=rng.choice(["bf16", "f16", "f32"]))
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 8, 8, 16])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    case = dict(op=op, seqs=_size(rng, 1, 64), T=0, ragged=rng.random() < 0.4, tree=rng.random() < 0.5, pad=rng.choice([0, 0, 1, 5]),
                lo=0, hi=0, heads=heads, kv=kv, d=d, type=kind, cache=rng.choice([kind, kind, "i8"]),
                page=rng.choice([16, 32, 48, 64, 256]))
    if op == "append":
        case.update(T=_size(rng, 1, 1500), hi=rng.choice([0, 300, 900]), rot=rng.choice([d, d, d // 2, d // 4 * 2 - 2]),
                    layout=rng.choice(["half", "pairs"]), norm=rng.random() < 0.6, amp=rng.choice([1.0, 1.2]),
                    type=rng.choice([kind, kind, "f32"]), out=kind)
        case["tree"] = case["tree"] and case["T"] <= 64
        return case
    case.update(T=rng.choice([1, 1, 2, 3, 4, 6, _size(rng, 5, 64)]), hi=_size(rng, 40, 131072), blank=rng.random() < 0.2)
    case["lo"] = rng.choice([0, case["hi"] // 3, case["hi"]])
    return case


def draw(rng):
    most = {}
    for case in listed():
        w = work(case)
        b, f = most.get(case["op"], (0, 0))
        most[case["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= most[case["op"]][0] and w["flops"] <= most[case["op"]][1] and w["flops"] > 0:
            return case


def _lengths(case):
    """The tokens of each sequence's window and its keys before them."""
    n = case["seqs"]
    tokens = [1 + (5 * s + case["T"] - 1) % case["T"] if case["ragged"] else case["T"] for s in range(n)]
    if case["ragged"] and n > 4:
        tokens[3] = 0
    return tokens, [case["lo"] + int((case["hi"] - case["lo"]) * ((0.618034 * s) % 1.0 if n > 1 else 1.0)) for s in range(n)]


def work(case):
    op = case["op"]
    if op == "logprobs":
        rows, n = case["rows"], case["n"]
        return {"bytes": rows * n * SIZE[case["type"]] + rows * (8 * case["given"] + 8 * case["k"] + 4 * case["entropy"]),
                "flops": rows * n * (6 if case["entropy"] else 4)}
    tokens, before = _lengths(case)
    H, kv, d, total = case["heads"], case["kv"], case["d"], sum(tokens)
    row = d * SIZE[case["cache"]] + (4 if case["cache"] == "i8" else 0)   # of the cache, its scale with it
    if op == "append":
        return {"bytes": total * ((H + 2 * kv) * d * SIZE[case["type"]] + H * d * SIZE[case["out"]] + 2 * kv * row),
                "flops": total * (H + kv) * (4 * d * case["norm"] + 3 * case["rot"])}
    keys = sum(t + b for t, b in zip(tokens, before) if t)
    pairs = sum(t * (t + b) for t, b in zip(tokens, before))
    return {"bytes": keys * kv * 2 * row + total * H * (2 * d * SIZE[case["type"]] + 4), "flops": 4 * pairs * H * d}


# ------------------------------------------------------------------ inputs ---------------------

def _trees(case, tokens, gen):
    """A tree for each sequence: token j's ancestors and itself as bits, and its depth."""
    seen, depth = [], []
    for t in tokens:
        pick = torch.rand(max(t, 1), generator=gen).tolist()
        bits, deep = [], []
        for j in range(t):
            parent = max(0, j - 1 - int(4 * pick[j])) if case["tree"] else j - 1
            bits.append(1 << j if j == 0 else bits[parent] | 1 << j)
            deep.append(0 if j == 0 else deep[parent] + 1)
        if case.get("blank"):   # padded places of the window: no token, nothing to see
            bits = [0 if j % 3 == 2 else b for j, b in enumerate(bits)]
        seen += [b - (1 << 64) if b >> 63 else b for b in bits]
        depth += deep
    return seen, depth


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    st, op = {"case": case}, case["op"]
    if op == "logprobs":
        rows, n = case["rows"], case["n"]
        # a few likely tokens above many unlikely ones; some rows sure of one
        x = 2.0 * randn(rows, n + case["extra"])
        x += 6.0 * (randn(1, n + case["extra"]) > 3.0) + randn(rows, 1)
        x[::5, n // 3] += 18.0
        if case["masked"]:   # a grammar's mask: most tokens of some rows, and every token of a padded row
            x.masked_fill_((randn(rows, 1) > 0.0) & (randn(1, n + case["extra"]) > -1.0), float("-inf"))
            x[rows // 2::17] = float("-inf")
        st["logits"] = x.to(DTYPES[case["type"]])[:, :n]
        st["tokens"] = torch.randint(0, n, (rows, case["given"]), generator=gen, device="cuda", dtype=torch.int32)
        if case["given"] > 2:
            st["tokens"][::3, 1] = -1   # nodes with fewer drafted tokens
        if own:
            _handles(st)
        return st
    tokens, before = _lengths(case)
    H, kv, d, page, n = case["heads"], case["kv"], case["d"], case["page"], sum(tokens)
    need = [(t + b + page - 1) // page for t, b in zip(tokens, before)]
    n_pages, cols = sum(need) + 2, max(max(need), 1)
    order, table, at = torch.randperm(n_pages, generator=host).tolist(), [], 0
    for count in need:
        table.append(order[at:at + count] + [-1] * (cols - count))
        at += count
    start = [0]
    for t in tokens:
        start.append(start[-1] + t)
    seen, depth = _trees(case, tokens, host)
    ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")
    st.update(row_start=ints(start), ctx_len=ints(before), pages=ints(table), n=n, tokens=tokens, before=before)
    st["seen"] = ints(seen + [0] * case["pad"], torch.int64) if case["tree"] or case.get("blank") else None
    shape = (n_pages, kv, page, d)
    if op == "append":
        st["pos"] = ints([b + e for b, e in zip([b for t, b in zip(tokens, before) for _ in range(t)], depth)] + [0] * case["pad"]) \
            if case["tree"] else None
        # the rows of one product, side by side; heads of different size
        part = torch.exp(0.4 * randn(H + 2 * kv)).repeat_interleave(d)
        st["qkv"] = (randn(n + case["pad"], (H + 2 * kv) * d) * part).to(DTYPES[case["type"]])
        t = DTYPES[case["type"]]
        st["q_weight"], st["k_weight"] = ((1.0 + 0.2 * randn(d)).to(t), (1.0 + 0.2 * randn(d)).to(t)) if case["norm"] else (None, None)
        # angles of a long context: the slow ones stretched
        i = torch.arange(case["rot"] // 2, dtype=torch.float64)
        f = 500000.0 ** (-2.0 * i / max(case["rot"], 1))
        st["freq"] = torch.where(f < 1e-3, f / 8.0, f).float().cuda()
        st["q_out"] = randn(n + case["pad"], H * d).to(DTYPES[case["out"]])
        if case["cache"] == "i8":
            st["k"], st["v"] = (torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8) for _ in range(2))
            st["k_scale"], st["v_scale"] = (0.01 * torch.exp(0.3 * randn(*shape[:3])) for _ in range(2))
        else:
            st["k"], st["v"] = randn(*shape).to(DTYPES[case["cache"]]), randn(*shape).to(DTYPES[case["cache"]])
    else:
        # some heads sharper than others
        st["q"] = (randn(n + case["pad"], H, d) * torch.exp(0.5 * randn(H, 1))).view(-1, H * d).to(DTYPES[case["type"]])
        st["out"] = randn(n + case["pad"], H * d).to(DTYPES[case["type"]])
        st["lse"] = randn(n + case["pad"], H)
        if case["cache"] == "i8":
            st["k"], st["v"] = (torch.round(40.0 * randn(*shape)).clamp_(-127, 127).to(torch.int8) for _ in range(2))
            st["k_scale"], st["v_scale"] = (0.025 * torch.exp(0.3 * randn(*shape[:3])) for _ in range(2))
        else:
            st["k"], st["v"] = randn(*shape).to(DTYPES[case["cache"]]), randn(*shape).to(DTYPES[case["cache"]])
    if own:
        _handles(st)
    return st


# ------------------------------------------------------------------ plain forms ----------------

def _places(st):
    """The page and slot of each window token, in order of tokens."""
    case = st["case"]
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device="cuda"), torch.tensor(st["tokens"], device="cuda"), output_size=st["n"])
    at = torch.arange(st["n"], device="cuda") - st["row_start"].long()[seq] + st["ctx_len"].long()[seq]
    return st["pages"].long()[seq, at // case["page"]], at % case["page"], at


def _int8(y):
    """int8 codes and float32 scales of float32 rows y: the quotient in float32, halves away from zero."""
    d = y.abs().amax(-1, keepdim=True)
    d = d / torch.full_like(d, 127.0)   # by a number, torch multiplies by its rounded reciprocal
    v = (y / torch.where(d > 0, d, torch.ones_like(d))).double()
    return (torch.sign(v) * torch.floor(v.abs() + 0.5).clamp_(max=127.0)).to(torch.int8), d.squeeze(-1)


def _plain_append(st):
    case, n = st["case"], st["n"]
    H, kv, d, rot = case["heads"], case["kv"], case["d"], case["rot"]
    page, slot, at = _places(st)
    # 64 bits: angles of far positions, and values next to a code's border
    x = st["qkv"][:n].double().view(n, H + 2 * kv, d)
    q, k, v = x[:, :H], x[:, H:H + kv], x[:, H + kv:]
    angle = (st["pos"][:n].double() if st["pos"] is not None else at.double())[:, None, None] * st["freq"].double()
    cos, sin = torch.cos(angle) * case["amp"], torch.sin(angle) * case["amp"]

    def turned(y, weight):
        if weight is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.double()
        y = y.clone()
        a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if case["layout"] == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
        a1, b1 = a * cos - b * sin, b * cos + a * sin
        a.copy_(a1)
        b.copy_(b1)
        return y.float()

    st["q_out"][:n] = turned(q, st["q_weight"]).view(n, -1).to(st["q_out"].dtype)
    out = {"q": st["q_out"]}
    for name, y in (("k", turned(k, st["k_weight"])), ("v", v.float())):
        pool = st[name]
        if case["cache"] == "i8":
            pool[page, :, slot], st[name + "_scale"][page, :, slot] = _int8(y)
            out[name] = pool.float() * st[name + "_scale"][..., None]
        else:
            pool[page, :, slot] = y.to(pool.dtype)
            out[name] = pool
    return out


def _plain_attend(st):
    case = st["case"]
    H, kv, d, size = case["heads"], case["kv"], case["d"], case["page"]
    G, row = H // kv, 0
    for s, (t, before) in enumerate(zip(st["tokens"], st["before"])):
        if not t:
            continue
        length = before + t
        pages = st["pages"][s, :(length + size - 1) // size].long()

        def keys(name):   # [kv, length, d]
            x = st[name][pages].float()
            if case["cache"] == "i8":
                x = x * st[name + "_scale"][pages][..., None]
            return x.transpose(0, 1).reshape(kv, -1, d)[:, :length]

        q = st["q"][row:row + t].float().view(t, kv, G, d).permute(1, 0, 2, 3).reshape(kv, t * G, d)
        scores = torch.matmul(q, keys("k").transpose(1, 2).contiguous()) * (d ** -0.5)
        j = torch.arange(t, device="cuda")
        if st["seen"] is not None:
            visible = (st["seen"][row:row + t, None] >> j) & 1 != 0
        else:
            visible = j[None, :] <= j[:, None]
        scores[:, :, before:].masked_fill_(~visible.repeat_interleave(G, 0), float("-inf"))
        top = scores.amax(-1, keepdim=True)
        top = top.masked_fill(torch.isneginf(top), 0.0)
        p = torch.exp(scores - top)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, keys("v").contiguous()) / total.masked_fill(total == 0, 1.0)
        st["out"][row:row + t] = o.view(kv, t, G, d).permute(1, 0, 2, 3).reshape(t, H * d).to(st["out"].dtype)
        st["lse"][row:row + t] = (torch.log(total) + top).view(kv, t, G).permute(1, 0, 2).reshape(t, H)
        row += t
    return {"out": st["out"], "lse": st["lse"]}


def _plain_logprobs(st):
    case = st["case"]
    x = st["logits"].float()
    if case["scale"] != 1.0:
        x = x * case["scale"]
    top = x.amax(-1, keepdim=True)
    top = top.masked_fill(torch.isneginf(top), 0.0)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True, dtype=torch.float64)   # 64 bits: a long sum
    log_total = torch.log(total)
    out = {}
    if case["given"]:
        at = st["tokens"].long()
        chosen = torch.gather(x, 1, at.clamp(min=0)) - top
        logp = torch.where(total > 0, chosen.double() - log_total, torch.full_like(log_total, float("-inf")))
        out["logp"] = logp.masked_fill(at < 0, float("-inf")).float()
    if case["entropy"]:
        mean = torch.where(e > 0, e * (x - top), torch.zeros_like(e)).sum(-1, keepdim=True, dtype=torch.float64)
        out["entropy"] = torch.where(total > 0, log_total - mean / total, torch.zeros_like(total)).float().squeeze(-1)
    if case["k"]:
        ids = torch.sort(st["logits"].float(), dim=-1, descending=True, stable=True).indices[:, :case["k"]]
        best = (torch.gather(x, 1, ids) - top).double() - log_total
        out["ids"] = ids.int()
        out["top"] = torch.where(total > 0, best, torch.full_like(best, float("-inf"))).float()
    return out


# ------------------------------------------------------------------ the library's calls --------

def _handles(st):
    """What a program keeps next to its cache: the handles of the cache and of the window, and workspaces."""
    from moe_routed_expert_route_amd import binding as B
    case = st["case"]
    if case["op"] == "logprobs":
        st["ws"] = B.logprobs_workspace(case["rows"], case["n"], case["k"])
        return
    st["cache"] = B.KVCache(st["k"], st["v"], st.get("k_scale"), st.get("v_scale"))
    st["window"] = B.Window(st["row_start"], st["ctx_len"], st["pages"], st["n"] + case["pad"], max_window=case["T"],
                            pos=st.get("pos"), seen=st["seen"] if case["op"] == "attend" else None)
    if case["op"] == "attend":
        st["ws"] = B.window_workspace(st["cache"], st["window"], case["heads"])


def _own_append(st):
    from moe_routed_expert_route_amd import binding as B
    case = st["case"]
    wide, kv = case["heads"] * case["d"], case["kv"] * case["d"]
    qkv = st["qkv"]
    B.moe_window_append(st["cache"], st["window"], qkv[:, :wide], qkv[:, wide:wide + kv], qkv[:, wide + kv:], freq=st["freq"],
                        layout=B.ROPE_HALF if case["layout"] == "half" else B.ROPE_PAIRS, amp=case["amp"], q_weight=st["q_weight"],
                        k_weight=st["k_weight"], eps=EPS, q_out=st["q_out"])
    out = {"q": st["q_out"]}
    for name in ("k", "v"):
        out[name] = torch.mul(st[name], st[name + "_scale"][..., None]) if case["cache"] == "i8" else st[name]
    return out


def _own_attend(st):
    from moe_routed_expert_route_amd import binding as B
    B.moe_window_attention(st["cache"], st["window"], st["q"], st["case"]["d"] ** -0.5, out=st["out"], lse=st["lse"], ws=st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_logprobs(st):
    from moe_routed_expert_route_amd import binding as B
    case = st["case"]
    logp, entropy, ids, top = B.moe_token_logprobs(st["logits"], tokens=st["tokens"] if case["given"] else None, k=case["k"],
                                                   entropy=case["entropy"], scale=case["scale"], ws=st["ws"])
    out = {"logp": logp, "entropy": entropy, "ids": ids, "top": top}
    return {name: t for name, t in out.items() if t is not None}


def run(state):
    op = state["case"]["op"]
    if own:
        if "ws" not in state and "cache" not in state:
            _handles(state)
        return {"append": _own_append, "attend": _own_attend, "logprobs": _own_logprobs}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "logprobs": _plain_logprobs}[op](state)


# ------------------------------------------------------------------ in 64 bits -----------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "logprobs": _exact_logprobs}[case["op"]](case, st)


def _values(case, st, name):
    x = st[name].double()
    return x * st[name + "_scale"].double()[..., None] if case["cache"] == "i8" else x


def _exact_append(case, st):
    """Head by head, the rotation as a product of complex numbers."""
    H, kv, d, rot, n = case["heads"], case["kv"], case["d"], case["rot"], st["n"]
    x = st["qkv"].double()
    out = {"q": st["q_out"].double(), "k": _values(case, st, "k"), "v": _values(case, st, "v")}
    seq = [s for s, t in enumerate(st["tokens"]) for _ in range(t)]
    at = [b + j for t, b in zip(st["tokens"], st["before"]) for j in range(t)]
    table = st["pages"].tolist()
    page = torch.tensor([table[s][a // case["page"]] for s, a in zip(seq, at)], device="cuda")
    slot = torch.tensor([a % case["page"] for a in at], device="cuda")
    where = st["pos"][:n].double() if st["pos"] is not None else torch.tensor(at, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full((n, rot // 2), case["amp"], dtype=torch.float64, device="cuda"), torch.outer(where, st["freq"].double()))
    first = torch.arange(rot // 2, device="cuda") * (1 if case["layout"] == "half" else 2)
    second = first + (rot // 2 if case["layout"] == "half" else 1)
    for h in range(H + 2 * kv):
        y = x[:n, h * d:(h + 1) * d].clone()
        if h < H + kv:
            weight = st["q_weight"] if h < H else st["k_weight"]
            if weight is not None:
                y *= (weight.double()[None] / torch.linalg.vector_norm(y, dim=1, keepdim=True).square().div(d).add(EPS).sqrt())
            z = torch.complex(y[:, first], y[:, second]) * turn
            y[:, first], y[:, second] = z.real, z.imag
        if h < H:
            out["q"][:n, h * d:(h + 1) * d] = y
            continue
        name, head = ("k", h - H) if h < H + kv else ("v", h - H - kv)
        if case["cache"] == "i8":   # the definition's own roundings: float32 rows, their scale, the quotient
            y = y.float()
            scale = y.abs().max(dim=1).values
            scale = torch.div(scale, torch.tensor(127.0, device="cuda").expand_as(scale))
            quotient = torch.where(scale[:, None] > 0, y / scale[:, None], torch.zeros_like(y)).double()
            whole = torch.trunc(quotient)
            code = whole + torch.where((quotient - whole).abs() >= 0.5, torch.sign(quotient), torch.zeros_like(whole))
            y = code.clamp(-127, 127) * scale.double()[:, None]
        out[name][page, head, slot] = y
    return out


def _exact_attend(case, st):
    """Token by token of the window and head by head, each over the keys that it sees."""
    H, kv, d, size = case["heads"], case["kv"], case["d"], case["page"]
    out, lse, row = st["out"].double(), st["lse"].double(), 0
    seen = st["seen"].tolist() if st["seen"] is not None else None
    for s, (t, before) in enumerate(zip(st["tokens"], st["before"])):
        if not t:
            continue
        at = torch.arange(before + t, device="cuda")
        page, slot = st["pages"][s].long()[at // size], at % size
        visible = torch.ones(t, before + t, dtype=torch.bool)
        for i in range(t):
            for j in range(t):
                visible[i, before + j] = bool(seen[row + i] >> j & 1) if seen is not None else j <= i
        visible = visible.cuda()
        for h in range(kv):
            K, V = st["k"][page, h, slot].double(), st["v"][page, h, slot].double()
            if case["cache"] == "i8":
                K *= st["k_scale"][page, h, slot].double()[:, None]
                V *= st["v_scale"][page, h, slot].double()[:, None]
            for g in range(h * (H // kv), (h + 1) * (H // kv)):
                score = (st["q"][row:row + t, g * d:(g + 1) * d].double() @ K.t()) / math.sqrt(d)
                score = torch.where(visible, score, torch.full_like(score, -math.inf))
                total = torch.logsumexp(score, dim=1)
                weight = torch.exp(score - total.masked_fill(torch.isneginf(total), 0.0)[:, None])
                out[row:row + t, g * d:(g + 1) * d] = weight @ V
                lse[row:row + t, g] = total
        row += t
    return {"out": out, "lse": lse}


def _exact_logprobs(case, st):
    rows, n = case["rows"], case["n"]
    bits = {"f32": torch.int32, "bf16": torch.int16, "f16": torch.int16}[case["type"]]
    parts = {"logp": [], "entropy": [], "ids": [], "top": []}
    for r in range(0, rows, 128):
        raw = st["logits"][r:r + 128]
        p = torch.log_softmax(raw.double() * case["scale"], dim=1)
        none = torch.isneginf(raw).all(dim=1, keepdim=True)
        p = p.masked_fill(none, -math.inf)
        at = st["tokens"][r:r + 128].long()
        parts["logp"].append(torch.gather(p, 1, at.clamp(min=0)).masked_fill(at < 0, -math.inf))
        parts["entropy"].append(-(torch.exp(p) * p.clamp(min=-1e30)).sum(1))
        if case["k"]:
            # one whole number for a value and its place: larger values first, then lower places
            v = (raw + 0.0).contiguous().view(bits).long()
            order = torch.where(v < 0, (-1 << 31 if case["type"] == "f32" else -1 << 15) - v, v)
            key = order * (1 << 20) + ((1 << 20) - 1 - torch.arange(n, device="cuda"))
            ids = torch.topk(key, case["k"], dim=1, sorted=True).indices
            parts["ids"].append(ids.int())
            parts["top"].append(torch.gather(p, 1, ids))
    wanted = {"logp": case["given"], "entropy": case["entropy"], "ids": case["k"], "top": case["k"]}
    return {name: torch.cat(part) for name, part in parts.items() if wanted[name]}
