"""Windows of tokens over a paged cache for tests, and the operators on them in 64 bits (numpy), one row and key at a time
where the size allows."""
import numpy as np
import torch

from moe_routed_expert_route_amd import binding as B
from moe_routed_expert_route_amd import synth

F32, BF16, F16, I8 = torch.float32, torch.bfloat16, torch.float16, torch.int8
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (F32, BF16, F16)}
TINY = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}   # a step of the smallest values
DEV = "cuda:0"


def host(t):
    return t.detach().cpu().double().numpy()


class Place:
    """Sequences of `tokens` after `ctx` keys, their pages dealt out in no order."""

    def __init__(self, tokens, ctx, n_kv=2, d=64, page=16, cache=BF16, key=0, pad=0, order="heads", seen=None, pos=None,
                 max_window=None, spare=2, table_pad=1):
        self.tokens, self.ctx, self.n_kv, self.d, self.page, self.dtype = list(tokens), list(ctx), n_kv, d, page, cache
        rng = synth.rng(key, 77)
        need = [-(-(t + c) // page) for t, c in zip(tokens, ctx)]
        self.n_pages = sum(need) + spare
        order_of = rng.permutation(self.n_pages)
        self.table = np.full((len(need), max(max(need), 1) + table_pad), -7, np.int32)
        at = 0
        for s, c in enumerate(need):
            self.table[s, :c] = order_of[at:at + c]
            at += c
        self.start = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
        self.n = int(self.start[-1])
        self.rows = self.n + pad
        self.seen_bits, self.pos = seen, pos

        def pool(scale):
            if cache is I8:
                x = torch.from_numpy(rng.integers(-127, 128, (self.n_pages, n_kv, page, d)).astype(np.int8))
            else:
                x = torch.from_numpy(scale * rng.standard_normal((self.n_pages, n_kv, page, d))).to(cache)
            if order == "slots":     # a slot's heads side by side
                return x.to(DEV).transpose(1, 2).contiguous().transpose(1, 2)
            if order == "wide":      # gaps between rows, heads and pages
                buf = torch.full((self.n_pages, n_kv + 1, page + 1, d + 16), 77, dtype=x.dtype, device=DEV)
                buf[:, :n_kv, :page, :d] = x.to(DEV)
                return buf[:, :n_kv, :page, :d]
            return x.to(DEV)

        self.k, self.v = pool(1.0), pool(1.0)
        if order == "both":          # keys and values of a page in one buffer
            buf = torch.stack([self.k, self.v], 1).contiguous()
            self.k, self.v = buf[:, 0], buf[:, 1]
        scales = (None, None)
        if cache is I8:
            scales = tuple(torch.from_numpy((0.02 * np.exp(0.3 * rng.standard_normal((self.n_pages, n_kv, page)))).astype(np.float32)).to(DEV)
                           for _ in range(2))
        self.k_scale, self.v_scale = scales
        self.cache = B.KVCache(self.k, self.v, *scales)
        ints = lambda v, t=torch.int32: torch.from_numpy(np.asarray(v)).to(t).to(DEV)
        wide = torch.full((self.table.shape[0], self.table.shape[1] + 3), -9, dtype=torch.int32, device=DEV)
        wide[:, :self.table.shape[1]] = ints(self.table)
        self.seen = None
        if seen is not None:
            bits = list(seen) + [0] * pad
            self.seen = torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device=DEV)
        self.window = B.Window(ints(self.start), ints(ctx), wide[:, :self.table.shape[1]], self.rows,
                               max_window=max_window or max(max(self.tokens), 1), seen=self.seen,
                               pos=None if pos is None else ints(list(pos) + [0] * pad))

    def key_at(self, s, i):
        """Page and slot of a sequence's key i."""
        return self.table[s, i // self.page], i % self.page

    def keys(self, s, h):
        """A sequence's keys and values of head h, in 64 bits."""
        at = np.arange(self.ctx[s] + self.tokens[s])
        page, slot = torch.from_numpy(self.table[s][at // self.page]).long().to(DEV), torch.from_numpy(at % self.page).to(DEV)
        out = []
        for pool, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            x = host(pool[page, h, slot])
            if scale is not None:
                x = x * host(scale[page, h, slot])[:, None]
            out.append(x)
        return out

    def sees(self, s, j):
        """The keys that token j of sequence s sees."""
        bits = self.seen_bits[self.start[s] + j] if self.seen_bits is not None else (2 << j) - 1
        return np.array([True] * self.ctx[s] + [bool(bits >> i & 1) for i in range(self.tokens[s])], dtype=bool)


def tree(tokens, key=0):
    """Bits of a random tree over the tokens of each sequence, and each token's depth."""
    rng, bits, depth = synth.rng(key, 78), [], []
    for t in tokens:
        mine, deep = [], []
        for j in range(t):
            parent = int(rng.integers(max(0, j - 5), j)) if j else -1
            mine.append((mine[parent] if j else 0) | 1 << j)
            deep.append(deep[parent] + 1 if j else 0)
        bits += mine
        depth += deep
    return bits, depth


def attend_ref(p, q, n_heads, scale, p_type=None, left_out=()):
    """out, lse and a bound of the error of each, in 64 bits: per row and head over the keys that it sees.

    The scores are sums of d products in float32 (each step off by 2^-24 of the sum of sizes, any order), scaled (two
    roundings) and put through exp2 (its argument off by 2^-23 of its size, itself by 2^-22): ds. A weight is rounded to
    q's type (half a step, u; below the type's normal numbers by far less than the sum's own error, since weights are kept
    2^14 above them); over an i8 cache a factor of its scale is rounded too (2^-23). Sums of n terms in float32 are off by n 2^-24
    of the sum of sizes, here of the weights and of weights times values; joining runs adds some roundings (16 allowed)."""
    G, u = n_heads // p.n_kv, HALF_STEP[q.dtype]
    x = host(q)
    out = np.zeros((p.n, n_heads * p.d))
    lse = np.full((p.n, n_heads), -np.inf)
    out_tol, lse_tol = np.zeros_like(out), np.zeros_like(lse)
    for s, t in enumerate(p.tokens):
        for h in range(p.n_kv):
            K, V = p.keys(s, h) if t else (None, None)
            for j in range(t):
                live = p.sees(s, j)
                for o in left_out:
                    if o[0] == s:
                        live[o[1]:o[2]] = False
                if not live.any():
                    continue
                k, v, row = K[live], V[live], p.start[s] + j
                for g in range(h * G, (h + 1) * G):
                    qq = x[row, g * p.d:(g + 1) * p.d]
                    sc = k @ qq * scale
                    top = sc.max()
                    e = np.exp(sc - top)
                    n = len(sc)
                    ds = (p.d + 6) * 2.0 ** -24 * (np.abs(k) @ np.abs(qq) * abs(scale)) + (np.abs(sc - top) + np.abs(sc)) * 2.0 ** -22 + 2.0 ** -21
                    w = e / e.sum()
                    out[row, g * p.d:(g + 1) * p.d] = w @ v
                    lse[row, g] = top + np.log(e.sum())
                    rel = (n + 16) * 2.0 ** -24
                    from_sum = (w * ds).sum() + rel
                    out_tol[row, g * p.d:(g + 1) * p.d] = (w * (u + 2.0 ** -22 + 2 * ds + rel)) @ np.abs(v) + from_sum * np.abs(w @ v)
                    lse_tol[row, g] = from_sum + 2.0 ** -22 * (np.abs(top) + np.log(n) + 1)
    out_tol += np.abs(out) * u + TINY[q.dtype]
    return out, lse, out_tol, lse_tol
