"""Python binding of libmoe_route.so: the C-ABI entry points under the same names.

Argument marshalling only: torch tensors supply device memory and the current HIP stream; every
step of the computation runs in the library's HIP kernels. If the library is not built the
functions raise (there is no fallback of any kind).
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_route.so")

Q8_0, NL4, CB2, CB3, Q5_1, NL4X = 1, 2, 3, 4, 5, 6
BLOCK_BYTES = {Q8_0: 34, NL4: 18, CB2: 70, CB3: 110, Q5_1: 24, NL4X: 136}
BLOCK_WEIGHTS = {Q8_0: 32, NL4: 32, CB2: 256, CB3: 256, Q5_1: 32, NL4X: 256}

ERR_BITS = {1: "NGROUPS", 2: "ENTRIES", 4: "EXPERT", 8: "SRC", 16: "DST", 32: "ALIGN", 64: "WAIT", 128: "WINDOW",
            256: "PAGE"}

EXPORTS = ("moe_route_topk", "moe_build_plan", "moe_quantize_q8_1", "moe_repack", "moe_gate_up",
           "moe_swiglu_q8_1", "moe_down_scatter", "moe_workspace_bytes",
           "moe_layer_decode", "moe_layer_decode_routed", "moe_layer_decode_routed_noalloc", "moe_layer_step", "moe_layer_gate_up",
           "moe_layer_down",
           "moe_workspace_layout", "moe_prefill_plan", "moe_prefill_gate_up", "moe_prefill_swiglu_q8_1",
           "moe_prefill_down", "moe_prefill_scatter",
           "moe_add_rmsnorm", "moe_route_scores", "moe_swiglu_i8", "moe_matmul_i8",
           "moe_window_append", "moe_window_attention_bytes", "moe_window_attention", "moe_token_logprobs_bytes",
           "moe_token_logprobs", "moe_stream_read", "moe_status_string", "moe_last_error")

_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_F = ctypes.c_float


class MoeLayer(ctypes.Structure):
    _fields_ = [("n_embd", ctypes.c_int32), ("n_ff", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("fmt_gate_up", ctypes.c_int32), ("fmt_down", ctypes.c_int32),
                ("gate", _P), ("up", _P), ("down", _P),
                ("nl4_table", _P), ("cb2_grid", _P), ("cb3_grid", _P)]


class MoePlan(ctypes.Structure):
    _fields_ = [("cap_groups", ctypes.c_int32), ("cap_entries", ctypes.c_int32),
                ("n_groups", _P), ("grp_expert", _P), ("grp_start", _P), ("ent_src", _P),
                ("ent_dst", _P), ("ent_w", _P), ("err", _P)]


class MoeKvCache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_stride", _L), ("head_stride", _L),
                ("slot_stride", _L), ("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P)]


class MoeWindow(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("max_window", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("ld_pages", _L), ("row_start", _P), ("ctx_len", _P), ("pages", _P),
                ("pos", _P), ("seen", _P), ("err", _P)]


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_route_topk.argtypes = [_P, _P, _I, _I, _I, _P, _P]
        L.moe_build_plan.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, ctypes.POINTER(MoePlan)]
        L.moe_quantize_q8_1.argtypes = [_P, _P, _I, _I, _P]
        L.moe_repack.argtypes = [_P, _I, _P, ctypes.c_int64, _I, _P, _I]
        L.moe_gate_up.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan), _P, _I, _P,
                                  _P, _I, _I]
        L.moe_swiglu_q8_1.argtypes = [_P, ctypes.POINTER(MoePlan), _P, _P, _I, _I, _P, _P]
        L.moe_down_scatter.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan), _P, _P,
                                       _I, _I, _I]
        L.moe_workspace_bytes.argtypes = [ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan)]
        L.moe_workspace_bytes.restype = ctypes.c_size_t
        L.moe_layer_decode.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan), _P, _I,
                                       _P, _I, _I, _P, ctypes.c_size_t, _I]
        L.moe_layer_decode_routed.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan),
                                              _P, _I, _I, _P, _I, _P, _P, _I, _I, _P,
                                              ctypes.c_size_t, _I]
        L.moe_layer_decode_routed_noalloc.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan),
                                                      _P, _I, _I, _P, _I, _P, _P, _I, _I, _I]
        L.moe_layer_step.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan),
                                     _P, _I, _I, _P, _I, _P, _P, _I, _I, _P, ctypes.c_size_t, _I]
        L.moe_layer_gate_up.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan), _P, _I,
                                        _I, _P, _I, _P, _I, _P, ctypes.c_size_t, _I]
        L.moe_layer_down.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan), _P,
                                     ctypes.c_size_t, _I, _P, _I, _I, _I]
        L.moe_workspace_layout.argtypes = [ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan), _P]
        L.moe_prefill_plan.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, ctypes.POINTER(MoePlan), _P]
        L.moe_prefill_gate_up.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan), _P, _I, _P,
                                          _P, _I]
        L.moe_prefill_swiglu_q8_1.argtypes = [_P, ctypes.POINTER(MoePlan), _P, _P, _I, _I, _P, _P]
        L.moe_prefill_down.argtypes = [_P, ctypes.POINTER(MoeLayer), ctypes.POINTER(MoePlan), _P, _P, _I]
        L.moe_prefill_scatter.argtypes = [_P, ctypes.POINTER(MoePlan), _P, _P, _I, _I, _P, _I, _I, _P, _I, _I]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [_I]
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_stream_read.argtypes = [_P, _P, ctypes.c_uint64, _P, _I]
        L.moe_add_rmsnorm.argtypes = [_P, _I, _P, _L, _P, _L, _I, _P, _F, _I, _I, _P, _L, _I, _P, _L, _P, _L, _P, _P]
        L.moe_route_scores.argtypes = [_P, _I, _P, _L, _I, _I, _I, _I, _P, _I, _I, _I, _I, _F, _P, _P]
        L.moe_swiglu_i8.argtypes = [_P, _I, _P, _L, _P, _L, _I, _I, _P, _L, _P]
        L.moe_matmul_i8.argtypes = [_P, _P, _L, _P, _P, _L, _P, _I, _I, _I, _I, _P, _L, _I]
        both = [ctypes.POINTER(MoeKvCache), ctypes.POINTER(MoeWindow)]
        L.moe_window_append.argtypes = [_P, *both, _I, _P, _L, _P, _L, _P, _L, _I, _I, _P, _P, _F, _P, _I, _I, ctypes.c_double, _I,
                                        _P, _L]
        L.moe_window_attention_bytes.argtypes = [*both, _I]
        L.moe_window_attention_bytes.restype = ctypes.c_size_t
        L.moe_window_attention.argtypes = [_P, *both, _I, _P, _L, _I, _F, _P, _L, _P, _P, ctypes.c_size_t]
        L.moe_token_logprobs_bytes.argtypes = [_I, _I, _I]
        L.moe_token_logprobs_bytes.restype = ctypes.c_size_t
        L.moe_token_logprobs.argtypes = [_P, _I, _P, _L, _I, _I, _F, _P, _I, _P, _P, _I, _P, _P, _P, ctypes.c_size_t]
        _lib = L
    return _lib


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, what: str):
    if rc != 0:
        L = lib()
        msg = L.moe_status_string(rc).decode()
        extra = L.moe_last_error().decode() if rc in (-4, -5) else ""
        raise RuntimeError(f"{what}: {msg} ({rc}) {extra}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# ------------------------------------------------------------------ device-side objects -------

class Layer:
    """One layer's experts on the device: byte tensors per expert, device pointer arrays and the
    C struct. `gate`, `up`, `down` are lists of uint8 tensors (or host arrays, uploaded)."""

    def __init__(self, n_embd, n_ff, fmt_gate_up, fmt_down, gate, up, down, nl4=None, cb2=None,
                 cb3=None, device="cuda"):
        def dev(a, dtype=torch.uint8):
            if a is None:
                return None
            t = a if isinstance(a, torch.Tensor) else torch.from_numpy(a)
            return t.to(device=device, dtype=dtype).contiguous()
        self.gate = [dev(a) for a in gate]
        self.up = [dev(a) for a in up]
        self.down = [dev(a) for a in down]
        self.nl4 = dev(nl4, torch.int8)
        self.cb2 = dev(cb2)
        self.cb3 = dev(cb3)
        self.ptr_gate = torch.tensor([t.data_ptr() for t in self.gate], dtype=torch.int64, device=device)
        self.ptr_up = torch.tensor([t.data_ptr() for t in self.up], dtype=torch.int64, device=device)
        self.ptr_down = torch.tensor([t.data_ptr() for t in self.down], dtype=torch.int64, device=device)
        self.n_embd, self.n_ff = n_embd, n_ff
        self.fmt_gate_up, self.fmt_down = fmt_gate_up, fmt_down
        self.struct = MoeLayer(n_embd, n_ff, len(self.gate), fmt_gate_up, fmt_down,
                               self.ptr_gate.data_ptr(), self.ptr_up.data_ptr(),
                               self.ptr_down.data_ptr(),
                               self.nl4.data_ptr() if self.nl4 is not None else None,
                               self.cb2.data_ptr() if self.cb2 is not None else None,
                               self.cb3.data_ptr() if self.cb3 is not None else None)

    @classmethod
    def from_pointers(cls, n_embd, n_ff, fmt_gate_up, fmt_down, ptr_gate, ptr_up, ptr_down,
                      nl4=None, cb2=None, cb3=None, keep=()):
        """Experts already resident elsewhere (e.g. a pool); ptr_* are int64 device tensors."""
        self = cls.__new__(cls)
        self.gate = self.up = self.down = []
        self.nl4, self.cb2, self.cb3 = nl4, cb2, cb3
        self.ptr_gate, self.ptr_up, self.ptr_down = ptr_gate, ptr_up, ptr_down
        self._keep = keep
        self.n_embd, self.n_ff = n_embd, n_ff
        self.fmt_gate_up, self.fmt_down = fmt_gate_up, fmt_down
        self.struct = MoeLayer(n_embd, n_ff, int(ptr_gate.numel()), fmt_gate_up, fmt_down,
                               ptr_gate.data_ptr(), ptr_up.data_ptr(), ptr_down.data_ptr(),
                               nl4.data_ptr() if nl4 is not None else None,
                               cb2.data_ptr() if cb2 is not None else None,
                               cb3.data_ptr() if cb3 is not None else None)
        return self


class Plan:
    """Device arrays of a call's plan. Entry arrays hold `entry_capacity` entries (absolute
    indices), so a plan may start past entry 0."""

    def __init__(self, cap_groups, cap_entries, entry_capacity=None, device="cuda", entries_of=None):
        """entries_of: another Plan whose entry arrays (and error word) this one shares, so that
        two calls of one layer (each over its own groups) index one run of entries."""
        ec = entry_capacity if entry_capacity is not None else cap_entries
        i32 = dict(dtype=torch.int32, device=device)
        self.n_groups = torch.zeros(1, **i32)
        self.grp_expert = torch.zeros(cap_groups, **i32)
        self.grp_start = torch.zeros(cap_groups + 1, **i32)
        if entries_of is not None:
            self.ent_src, self.ent_dst = entries_of.ent_src, entries_of.ent_dst
            self.ent_w, self.err = entries_of.ent_w, entries_of.err
        else:
            self.ent_src = torch.zeros(ec, **i32)
            self.ent_dst = torch.zeros(ec, **i32)
            self.ent_w = torch.zeros(ec, dtype=torch.float32, device=device)
            self.err = torch.zeros(1, **i32)
        self.cap_groups, self.cap_entries = cap_groups, cap_entries
        self.struct = MoePlan(cap_groups, cap_entries, self.n_groups.data_ptr(),
                              self.grp_expert.data_ptr(), self.grp_start.data_ptr(),
                              self.ent_src.data_ptr(), self.ent_dst.data_ptr(),
                              self.ent_w.data_ptr(), self.err.data_ptr())

    def set(self, plan: dict):
        """Copy a host plan (dict of numpy arrays with absolute entry indices) in."""
        ng = int(plan["n_groups"])
        base = int(plan["entry_base"])
        self.n_groups.fill_(ng)
        if ng:
            self.grp_expert[:ng].copy_(torch.as_tensor(plan["grp_expert"][:ng], dtype=torch.int32))
        self.grp_start[:ng + 1].copy_(torch.as_tensor(plan["grp_start"][:ng + 1], dtype=torch.int32))
        n = len(plan["ent_src"])
        if n:
            self.ent_src[base:base + n].copy_(torch.as_tensor(plan["ent_src"], dtype=torch.int32))
            self.ent_dst[base:base + n].copy_(torch.as_tensor(plan["ent_dst"], dtype=torch.int32))
            self.ent_w[base:base + n].copy_(torch.as_tensor(plan["ent_w"], dtype=torch.float32))

    def get(self) -> dict:
        """Host copy (synchronises)."""
        ng = int(self.n_groups.item())
        gs = self.grp_start[:ng + 1].cpu().numpy()
        base = int(gs[0]) if ng else 0
        end = int(gs[-1]) if ng else 0
        return dict(n_groups=ng, grp_expert=self.grp_expert[:ng].cpu().numpy(), grp_start=gs,
                    entry_base=base, ent_src=self.ent_src[base:end].cpu().numpy(),
                    ent_dst=self.ent_dst[base:end].cpu().numpy(),
                    ent_w=self.ent_w[base:end].cpu().numpy())

    def errors(self) -> int:
        return int(self.err.item()) & 0xFFFFFFFF


# ------------------------------------------------------------------ entry points --------------

LAYOUT_PLANAR = 0x100   # OR-ed into a layer's format field: planar rows (see moe_repack)


def moe_repack(fmt, src, rows, cols, dst=None, to_planar=True, stream=None):
    """rows x cols weights of base format `fmt` (uint8 device tensor `src`) into the planar layout
    (to_planar) or back into the row-major one; returns dst (a new tensor unless given)."""
    dst = dst if dst is not None else torch.empty_like(src)
    _check(lib().moe_repack(_stream(stream), int(fmt), _ptr(src), int(rows), int(cols), _ptr(dst),
                            1 if to_planar else 0), "moe_repack")
    return dst


# ------------------------------------------------------------------ prompt path ---------------

def moe_prefill_plan(ids, w, plan: Plan, E, dst_of_token=None, entry_base=0, ent_of=None, stream=None):
    """Plan of T x k choices (ids, w int32 / float32 [T, k] device tensors); returns ent_of [T, k]."""
    T, k = ids.shape
    ent_of = ent_of if ent_of is not None else torch.empty((T, k), dtype=torch.int32, device=ids.device)
    _check(lib().moe_prefill_plan(_stream(stream), _ptr(ids), _ptr(w), _ptr(dst_of_token), T, k, E,
                                  entry_base, ctypes.byref(plan.struct), _ptr(ent_of)), "moe_prefill_plan")
    return ent_of


def moe_prefill_gate_up(layer: Layer, plan: Plan, xq, g, u, stream=None):
    _check(lib().moe_prefill_gate_up(_stream(stream), ctypes.byref(layer.struct), ctypes.byref(plan.struct),
                                     _ptr(xq), xq.shape[0], _ptr(g), _ptr(u), g.stride(0)),
           "moe_prefill_gate_up")


def moe_prefill_swiglu_q8_1(plan: Plan, g, u, n_ff, hq, h=None, stream=None):
    _check(lib().moe_prefill_swiglu_q8_1(_stream(stream), ctypes.byref(plan.struct), _ptr(g), _ptr(u), n_ff,
                                         g.stride(0), _ptr(h), _ptr(hq)), "moe_prefill_swiglu_q8_1")


def moe_prefill_down(layer: Layer, plan: Plan, hq, O, stream=None):
    _check(lib().moe_prefill_down(_stream(stream), ctypes.byref(layer.struct), ctypes.byref(plan.struct),
                                  _ptr(hq), _ptr(O), O.stride(0)), "moe_prefill_down")


def moe_prefill_scatter(plan: Plan, ent_of, O, Y, n_embd, dst_of_token=None, stream=None):
    T, k = ent_of.shape
    _check(lib().moe_prefill_scatter(_stream(stream), ctypes.byref(plan.struct), _ptr(ent_of),
                                     _ptr(dst_of_token), T, k, _ptr(O), O.stride(0), n_embd, _ptr(Y),
                                     Y.shape[0], Y.stride(0)), "moe_prefill_scatter")


def moe_route_topk(logits, k, ids=None, w=None, stream=None):
    T, E = logits.shape
    ids = ids if ids is not None else torch.empty((T, k), dtype=torch.int32, device=logits.device)
    w = w if w is not None else torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(lib().moe_route_topk(_stream(stream), _ptr(logits), T, E, k, _ptr(ids), _ptr(w)),
           "moe_route_topk")
    return ids, w


def moe_build_plan(ids, w, plan: Plan, E, dst_of_token=None, entry_base=0, stream=None):
    T, k = ids.shape
    _check(lib().moe_build_plan(_stream(stream), _ptr(ids), _ptr(w), _ptr(dst_of_token), T, k, E,
                                entry_base, ctypes.byref(plan.struct)), "moe_build_plan")


def moe_quantize_q8_1(x, q=None, stream=None):
    rows, n = x.shape
    q = q if q is not None else torch.empty((rows, n // 32 * 36), dtype=torch.uint8, device=x.device)
    _check(lib().moe_quantize_q8_1(_stream(stream), _ptr(x), rows, n, _ptr(q)), "moe_quantize_q8_1")
    return q


def moe_gate_up(layer: Layer, plan: Plan, xq, g, u, grid_limit=0, stream=None):
    _check(lib().moe_gate_up(_stream(stream), ctypes.byref(layer.struct), ctypes.byref(plan.struct),
                             _ptr(xq), xq.shape[0], _ptr(g), _ptr(u), g.stride(0), grid_limit),
           "moe_gate_up")


def moe_swiglu_q8_1(plan: Plan, g, u, n_ff, hq, h=None, stream=None):
    _check(lib().moe_swiglu_q8_1(_stream(stream), ctypes.byref(plan.struct), _ptr(g), _ptr(u), n_ff,
                                 g.stride(0), _ptr(h), _ptr(hq)), "moe_swiglu_q8_1")


def moe_workspace_bytes(layer: Layer, plan: Plan) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(layer.struct), ctypes.byref(plan.struct)))


def workspace(layer: Layer, plan: Plan, device="cuda"):
    """Allocate a zero-filled workspace for this layer geometry and plan capacity (the one-launch
    step needs its flags and counts zero before the first call; every other call reads only bytes
    it wrote itself)."""
    nb = moe_workspace_bytes(layer, plan)
    if nb == 0:
        raise RuntimeError("moe_workspace_bytes: bad layer or plan")
    ws = torch.zeros(nb, dtype=torch.uint8, device=device)
    if ws.data_ptr() % 256:
        raise RuntimeError("workspace not 256-byte aligned")
    return ws


def moe_workspace_layout(layer: Layer, plan: Plan):
    """Byte offsets of the split q8_1 rows of h in the workspace: low quant halves, high quant
    halves, float scales."""
    off = (ctypes.c_size_t * 3)()
    _check(lib().moe_workspace_layout(ctypes.byref(layer.struct), ctypes.byref(plan.struct), off),
           "moe_workspace_layout")
    return [int(v) for v in off]


def moe_down_scatter(layer: Layer, plan: Plan, hq, Y, grid_limit=0, stream=None):
    _check(lib().moe_down_scatter(_stream(stream), ctypes.byref(layer.struct), ctypes.byref(plan.struct),
                                  _ptr(hq), _ptr(Y), Y.shape[0], Y.stride(0), grid_limit),
           "moe_down_scatter")


def moe_layer_decode(layer: Layer, plan: Plan, x, Y, ws, grid_limit=0, stream=None):
    _check(lib().moe_layer_decode(_stream(stream), ctypes.byref(layer.struct), ctypes.byref(plan.struct),
                                  _ptr(x), x.shape[0], _ptr(Y), Y.shape[0], Y.stride(0), _ptr(ws),
                                  ws.numel(), grid_limit), "moe_layer_decode")


def moe_layer_decode_routed(layer: Layer, plan: Plan, logits, k, x, Y, ws, dst_of_token=None,
                            entry_base=0, grid_limit=0, stream=None):
    T = logits.shape[0]
    _check(lib().moe_layer_decode_routed(_stream(stream), ctypes.byref(layer.struct),
                                         ctypes.byref(plan.struct), _ptr(logits), T, k,
                                         _ptr(dst_of_token), entry_base, _ptr(x), _ptr(Y), Y.shape[0],
                                         Y.stride(0), _ptr(ws), ws.numel(), grid_limit),
           "moe_layer_decode_routed")


def moe_layer_decode_routed_noalloc(layer: Layer, plan: Plan, logits, k, x, Y, dst_of_token=None,
                                    entry_base=0, grid_limit=0, stream=None):
    """moe_layer_decode_routed with the library's static scratch as its workspace (nothing is
    allocated); calls that overlap on one GPU race."""
    T = logits.shape[0]
    _check(lib().moe_layer_decode_routed_noalloc(_stream(stream), ctypes.byref(layer.struct),
                                                 ctypes.byref(plan.struct), _ptr(logits), T, k,
                                                 _ptr(dst_of_token), entry_base, _ptr(x), _ptr(Y), Y.shape[0],
                                                 Y.stride(0), grid_limit),
           "moe_layer_decode_routed_noalloc")


def moe_layer_step(layer: Layer, plan: Plan, logits, k, x, Y, ws, dst_of_token=None, entry_base=0,
                   grid_limit=0, stream=None):
    """The whole step from the logits in one launch (workgroups meet through counts in ws)."""
    T = logits.shape[0]
    _check(lib().moe_layer_step(_stream(stream), ctypes.byref(layer.struct), ctypes.byref(plan.struct),
                                _ptr(logits), T, k, _ptr(dst_of_token), entry_base, _ptr(x), _ptr(Y),
                                Y.shape[0], Y.stride(0), _ptr(ws), ws.numel(), grid_limit),
           "moe_layer_step")


def moe_layer_gate_up(layer: Layer, plan: Plan, x, ws, logits=None, k=0, dst_of_token=None,
                      entry_base=0, grid_limit=0, stream=None):
    """First launch of the layer step (routing and grouping too when logits are given)."""
    T = logits.shape[0] if logits is not None else 0
    _check(lib().moe_layer_gate_up(_stream(stream), ctypes.byref(layer.struct), ctypes.byref(plan.struct),
                                   _ptr(logits), T, k, _ptr(dst_of_token), entry_base, _ptr(x),
                                   x.shape[0], _ptr(ws), ws.numel(), grid_limit), "moe_layer_gate_up")


def moe_layer_down(layer: Layer, plan: Plan, ws, n_tokens, Y, grid_limit=0, stream=None):
    """Second launch of the layer step: down over the workspace's h rows + scatter into Y."""
    _check(lib().moe_layer_down(_stream(stream), ctypes.byref(layer.struct), ctypes.byref(plan.struct),
                                _ptr(ws), ws.numel(), n_tokens, _ptr(Y), Y.shape[0], Y.stride(0),
                                grid_limit), "moe_layer_down")


# ------------------------------------------------------------------ around the layer ----------

F32, BF16, F16 = 1, 2, 3                 # element types of rows (moe_dtype)
SCORE_SOFTMAX, SCORE_SIGMOID = 1, 2      # moe_score
_DTYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


_FLOATS, _INT8, _F32ONLY, _BYTES, _INT32 = tuple(_DTYPE), (torch.int8,), (torch.float32,), (torch.uint8,), (torch.int32,)
_HALVES = (torch.bfloat16, torch.float16)


# These calls can be a few microseconds long: the checks below ask each tensor for as little as they can,
# pointers go to ctypes as plain numbers, and the stream comes without a Stream object.
def _call(what, device, *args):
    """Enqueues on the current stream of the tensors' GPU `device` (an index), with that GPU current."""
    st = torch._C._cuda_getCurrentRawStream(device)
    fn = getattr(_lib or lib(), what)
    if torch._C._cuda_getDevice() == device:
        rc = fn(st, *args)
    else:
        with torch.cuda.device(device):
            rc = fn(st, *args)
    if rc:
        _check(rc, what)


def _on(stream, f, *args):
    """f(*args), and what it allocates, on `stream`."""
    device = args[0].get_device()
    if device >= 0 and stream.device_index != device:
        raise ValueError(f"{f.__name__}: the stream is of GPU {stream.device_index}, the tensors are on {device}")
    with torch.cuda.stream(stream):
        return f(*args)


def _on_cache(stream, f, cache, *args):
    """f(cache, *args), and what it allocates, on `stream`."""
    if stream.device_index != cache.device:
        raise ValueError(f"{f.__name__}: the stream is of GPU {stream.device_index}, the cache is on {cache.device}")
    with torch.cuda.stream(stream):
        return f(cache, *args)


def _gpu(what, name, t):
    """The index of the GPU that t, the call's first tensor, is on."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{what}: {name} is on {t.device}, not on a GPU")
    return device


def _rows(what, name, t, shape, dtypes, device):
    """The row stride of t, checked to be rows (any stride, elements next to each other) of `shape` (None:
    any) and one of `dtypes` on GPU `device`."""
    size = t.shape
    if len(size) != 2 or (shape is not None and size != shape):
        raise ValueError(f"{what}: {name} has shape {tuple(size)}, not " + ("rows" if shape is None else str(tuple(shape))))
    if shape is None and (size[0] | size[1]) >> 31:
        raise ValueError(f"{what}: {name} has shape {tuple(size)}, past 32 bits")
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: {name} is {t.dtype}, not one of {dtypes}")
    if t.get_device() != device:
        raise ValueError(f"{what}: {name} is on {t.device}, not on the call's GPU")
    if t.is_contiguous():
        return size[1]
    rows, n = size
    ld, step = t.stride()
    if step != 1 and n > 1:
        raise ValueError(f"{what}: {name}'s row elements are not next to each other")
    return ld if rows > 1 or ld > n else n


def _packed(what, name, t, shape, dtype, device):
    """t checked to be contiguous, of `shape` and `dtype` on GPU `device`."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: {name} is {t.dtype} {tuple(t.shape)} on {t.device}, not contiguous {dtype} {shape} on the "
                         "call's GPU")


def i8_rows(rows, n, device="cuda"):
    """New int8 rows and their scales: q [rows, n] (rows 16-byte aligned), scale [rows] float32."""
    q = torch.empty((rows, (n + 15) // 16 * 16), dtype=torch.int8, device=device)
    return (q if n % 16 == 0 else q[:, :n]), torch.empty(rows, dtype=torch.float32, device=device)


def moe_add_rmsnorm(x, weight, eps, res=None, res_out=None, y=None, q=None, scale=None, q8_1=None, stream=None):
    """RMS norm of x (+ res) rows [rows, n] into the outputs given: res_out (the sum, may be x or
    res), y (float rows), q and scale (int8 rows), q8_1 (uint8 [rows, n / 32 * 36])."""
    what = "moe_add_rmsnorm"
    if stream is not None:
        return _on(stream, moe_add_rmsnorm, x, weight, eps, res, res_out, y, q, scale, q8_1)
    dev, size, same = _gpu(what, "x", x), x.shape, (x.dtype,)
    ldx = _rows(what, "x", x, None, _FLOATS, dev)
    rows, n = size
    if weight.dtype not in _DTYPE:
        raise ValueError(f"{what}: weight is {weight.dtype}")
    _packed(what, "weight", weight, (n,), weight.dtype, dev)
    ldres = ldro = ldy = ldq = y_type = 0
    if res is not None:
        ldres = _rows(what, "res", res, size, same, dev)
    if res_out is not None:
        ldro = _rows(what, "res_out", res_out, size, same, dev)
    if y is not None:
        ldy, y_type = _rows(what, "y", y, size, _FLOATS, dev), _DTYPE[y.dtype]
    if q is not None:
        ldq = _rows(what, "q", q, size, _INT8, dev)
    if scale is not None:
        _packed(what, "scale", scale, (rows,), torch.float32, dev)
    if q8_1 is not None:
        if n % 32:
            raise ValueError(f"{what}: q8_1 rows need a multiple of 32 values, not {n}")
        _packed(what, "q8_1", q8_1, (rows, n // 32 * 36), torch.uint8, dev)
    _call(what, dev, _DTYPE[x.dtype], x.data_ptr(), ldx, res.data_ptr() if res is not None else 0, ldres,
          _DTYPE[weight.dtype], weight.data_ptr(), eps, rows, n, res_out.data_ptr() if res_out is not None else 0, ldro,
          y_type, y.data_ptr() if y is not None else 0, ldy, q.data_ptr() if q is not None else 0, ldq,
          scale.data_ptr() if scale is not None else 0, q8_1.data_ptr() if q8_1 is not None else 0)


def moe_route_scores(logits, k, score=SCORE_SOFTMAX, bias=None, n_groups=1, keep_groups=1, group_top=1, renorm=True,
                     factor=1.0, ids=None, w=None, stream=None):
    """The k experts of each token (int32 [T, k]) and their weights (float32 [T, k]) from logits [T, E]."""
    what = "moe_route_scores"
    if stream is not None:
        return _on(stream, moe_route_scores, logits, k, score, bias, n_groups, keep_groups, group_top, renorm, factor, ids, w)
    dev = _gpu(what, "logits", logits)
    ld = _rows(what, "logits", logits, None, _FLOATS, dev)
    T, E = logits.shape
    if not 0 < k <= E >= n_groups >= keep_groups > 0 < group_top <= E:
        raise ValueError(f"{what}: k {k}, groups {n_groups}, {keep_groups} kept by {group_top}, of {E} experts")
    if score != SCORE_SOFTMAX and score != SCORE_SIGMOID:
        raise ValueError(f"{what}: score {score}")
    if bias is not None:
        _packed(what, "bias", bias, (E,), torch.float32, dev)
    if ids is None:
        ids = logits.new_empty((T, k), dtype=torch.int32)
    else:
        _packed(what, "ids", ids, (T, k), torch.int32, dev)
    if w is None:
        w = logits.new_empty((T, k), dtype=torch.float32)
    else:
        _packed(what, "w", w, (T, k), torch.float32, dev)
    _call(what, dev, _DTYPE[logits.dtype], logits.data_ptr(), ld, T, E, k, score,
          bias.data_ptr() if bias is not None else 0, n_groups, keep_groups, group_top, 1 if renorm else 0, factor,
          ids.data_ptr(), w.data_ptr())
    return ids, w


def moe_swiglu_i8(g, u, q=None, scale=None, stream=None):
    """int8 rows (q, scale) of silu(g) * u for rows g, u [rows, n], each of its own row stride."""
    what = "moe_swiglu_i8"
    if stream is not None:
        return _on(stream, moe_swiglu_i8, g, u, q, scale)
    dev, size = _gpu(what, "g", g), g.shape
    ldg = _rows(what, "g", g, None, _FLOATS, dev)
    ldu = _rows(what, "u", u, size, (g.dtype,), dev)
    rows, n = size
    if (q is None) != (scale is None):
        raise ValueError(f"{what}: q and scale come together")
    if q is None:
        q, scale = i8_rows(rows, n, g.device)
        ldq = q.stride(0)
    else:
        ldq = _rows(what, "q", q, size, _INT8, dev)
        _packed(what, "scale", scale, (rows,), torch.float32, dev)
    _call(what, dev, _DTYPE[g.dtype], g.data_ptr(), ldg, u.data_ptr(), ldu, rows, n, q.data_ptr(), ldq,
          scale.data_ptr())
    return q, scale


def moe_matmul_i8(a, sa, b, sb, c=None, dtype=torch.float32, accumulate=False, stream=None):
    """C [M, N] (+)= (a [M, K] . b [N, K]^T) * sa [M] * sb [N] for int8 rows a, b; c, or a new tensor
    of `dtype`."""
    what = "moe_matmul_i8"
    if stream is not None:
        return _on(stream, moe_matmul_i8, a, sa, b, sb, c, dtype, accumulate)
    dev = _gpu(what, "a", a)
    lda, ldb = _rows(what, "a", a, None, _INT8, dev), _rows(what, "b", b, None, _INT8, dev)
    M, K = a.shape
    N, kb = b.shape
    if kb != K:
        raise ValueError(f"{what}: rows of {K} and of {kb} values")
    _packed(what, "sa", sa, (M,), torch.float32, dev)
    _packed(what, "sb", sb, (N,), torch.float32, dev)
    if c is None:
        if accumulate or dtype not in _DTYPE:
            raise ValueError(f"{what}: accumulate needs c" if accumulate else f"{what}: dtype {dtype}")
        c, ldc = a.new_empty((M, N), dtype=dtype), N
    else:
        dtype, ldc = c.dtype, _rows(what, "c", c, (M, N), _FLOATS, dev)
    _call(what, dev, a.data_ptr(), lda, sa.data_ptr(), b.data_ptr(), ldb, sb.data_ptr(), M, N, K, _DTYPE[dtype],
          c.data_ptr(), ldc, 1 if accumulate else 0)
    return c


# ------------------------------------------------------------------ windows over a cache ------

I8 = 4                                   # moe_kv_cache.dtype of int8 rows
ROPE_HALF, ROPE_PAIRS = 1, 2             # moe_rope
MAX_WINDOW = 64                          # tokens of one sequence in moe_window_attention
_CACHE_DTYPE = {torch.bfloat16: BF16, torch.float16: F16, torch.int8: I8}


class KVCache:
    """A layer's paged cache: k and v [n_pages, n_kv, page_size, head_dim] (bfloat16, float16 or int8; any strides of
    the first three, the same for both; a cache of another order is passed as its permuted view), and for int8 rows the
    scales k_scale and v_scale, contiguous float32 [n_pages, n_kv, page_size]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        what = "KVCache"
        self.device = _gpu(what, "k", k)
        if k.dim() != 4 or k.dtype not in _CACHE_DTYPE:
            raise ValueError(f"{what}: k is {k.dtype} {tuple(k.shape)}, not a cache [pages, heads, slots, head_dim]")
        if v.shape != k.shape or v.dtype is not k.dtype or v.get_device() != self.device or v.stride() != k.stride():
            raise ValueError(f"{what}: v is {v.dtype} {tuple(v.shape)} of strides {v.stride()}, not as k")
        if k.stride(3) != 1 or max(k.shape) >> 31:
            raise ValueError(f"{what}: strides {k.stride()} of {tuple(k.shape)}")
        if (k_scale is None) == (k.dtype is torch.int8) or (v_scale is None) == (k.dtype is torch.int8):
            raise ValueError(f"{what}: scales come with int8 rows, and they with scales")
        if k_scale is not None:
            _packed(what, "k_scale", k_scale, k.shape[:3], torch.float32, self.device)
            _packed(what, "v_scale", v_scale, k.shape[:3], torch.float32, self.device)
        self.k, self.v, self.k_scale, self.v_scale, self.dtype = k, v, k_scale, v_scale, k.dtype
        self.n_pages, self.n_kv, self.page_size, self.head_dim = k.shape
        self.struct = MoeKvCache(_CACHE_DTYPE[k.dtype], self.n_pages, self.page_size, self.n_kv, self.head_dim, *k.stride()[:3],
                                 k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if k_scale is not None else None,
                                 v_scale.data_ptr() if v_scale is not None else None)
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, n_pages, page_size, n_kv, head_dim, dtype, device="cuda"):
        """A new cache of zeros, a head's slots of a page side by side."""
        k, v = (torch.zeros((n_pages, n_kv, page_size, head_dim), dtype=dtype, device=device) for _ in range(2))
        if dtype is not torch.int8:
            return cls(k, v)
        return cls(k, v, *(torch.zeros((n_pages, n_kv, page_size), dtype=torch.float32, device=device) for _ in range(2)))


class Window:
    """The tokens of one call: row_start int32 [n_seqs + 1], ctx_len int32 [n_seqs], pages int32 [n_seqs, max_pages] (any
    row stride), the number of rows, the most tokens of one sequence (attention's tiles of rows go by it; if not given, as
    many as there are rows, of several sequences 64 at most, which is what attention takes), pos int32 [n_tokens]
    (rotary positions, if not the keys' indices) and seen int64 [n_tokens] (the tokens of its window that each sees, as
    bits, if not itself and those before it). The tensors are read when a call runs."""

    def __init__(self, row_start, ctx_len, pages, n_tokens, max_window=None, pos=None, seen=None):
        what = "Window"
        self.device, n = _gpu(what, "row_start", row_start), ctx_len.shape[0]
        _packed(what, "row_start", row_start, (n + 1,), torch.int32, self.device)
        _packed(what, "ctx_len", ctx_len, (n,), torch.int32, self.device)
        ld = _rows(what, "pages", pages, None, _INT32, self.device)
        if pages.shape[0] != n or not 0 <= n_tokens < 1 << 31:
            raise ValueError(f"{what}: pages of {pages.shape[0]} sequences, not {n}, or {n_tokens} rows")
        if pos is not None:
            _packed(what, "pos", pos, (n_tokens,), torch.int32, self.device)
        if seen is not None:
            _packed(what, "seen", seen, (n_tokens,), torch.int64, self.device)
        if max_window is None:
            max_window = max(1, n_tokens if n == 1 else min(n_tokens, MAX_WINDOW))
        if not 0 < max_window < 1 << 31:
            raise ValueError(f"{what}: max_window {max_window}")
        self.row_start, self.ctx_len, self.pages, self.pos, self.seen = row_start, ctx_len, pages, pos, seen
        self.n_seqs, self.n_tokens, self.max_window = n, n_tokens, max_window
        self.err = torch.zeros(1, dtype=torch.int32, device=row_start.device)
        self.struct = MoeWindow(n, n_tokens, max_window, pages.shape[1], ld, row_start.data_ptr(), ctx_len.data_ptr(),
                                pages.data_ptr(), pos.data_ptr() if pos is not None else None,
                                seen.data_ptr() if seen is not None else None, self.err.data_ptr())
        self.ref = ctypes.byref(self.struct)

    def errors(self) -> int:
        """The device's error word (sticky; ERR_BITS names the bits)."""
        return int(self.err.item())


def _over_cache(what, cache, window):
    if window.device != cache.device:
        raise ValueError(f"{what}: the window is on GPU {window.device}, the cache on {cache.device}")
    return cache.device


def moe_window_append(cache: KVCache, window: Window, q, k, v, freq=None, layout=ROPE_HALF, amp=1.0, q_weight=None,
                      k_weight=None, eps=1e-6, q_out=None, stream=None):
    """The window's keys and values (rows k, v [n_tokens, n_kv * head_dim]) into the cache, keys normed (k_weight) and
    rotated (freq float32 [n_rot / 2]); its queries (rows q [n_tokens, n_heads * head_dim] or None) normed and rotated
    into q_out, which is returned (new rows of q's type if None; it may be q)."""
    what = "moe_window_append"
    if stream is not None:
        return _on_cache(stream, moe_window_append, cache, window, q, k, v, freq, layout, amp, q_weight, k_weight, eps, q_out)
    dev, n, d = _over_cache(what, cache, window), window.n_tokens, cache.head_dim
    kv = (n, cache.n_kv * d)
    ldk, ldv = _rows(what, "k", k, kv, _FLOATS, dev), _rows(what, "v", v, kv, (k.dtype,), dev)
    ldq = ldo = n_heads = o_type = n_rot = w_type = 0
    if q is not None:
        ldq, wide = _rows(what, "q", q, None, (k.dtype,), dev), q.shape[1]
        n_heads = wide // d
        if q.shape[0] != n or wide % d:
            raise ValueError(f"{what}: q has shape {tuple(q.shape)}, not {n} rows of heads of {d}")
        if q_out is None:
            q_out, ldo = q.new_empty((n, wide)), wide
        else:
            ldo = _rows(what, "q_out", q_out, q.shape, _FLOATS, dev)
        o_type = _DTYPE[q_out.dtype]
    elif q_out is not None or q_weight is not None:
        raise ValueError(f"{what}: q_out and q_weight without q")
    if layout not in (ROPE_HALF, ROPE_PAIRS):
        raise ValueError(f"{what}: layout {layout}")
    if freq is not None:
        n_rot = 2 * freq.shape[0]
        _packed(what, "freq", freq, (n_rot // 2,), torch.float32, dev)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            if w.dtype not in _DTYPE or (w_type and _DTYPE[w.dtype] != w_type):
                raise ValueError(f"{what}: {name} is {w.dtype}")
            w_type = _DTYPE[w.dtype]
            _packed(what, name, w, (d,), w.dtype, dev)
    _call(what, dev, cache.ref, window.ref, _DTYPE[k.dtype], q.data_ptr() if q is not None else 0, ldq, k.data_ptr(), ldk,
          v.data_ptr(), ldv, n_heads, w_type, q_weight.data_ptr() if q_weight is not None else 0,
          k_weight.data_ptr() if k_weight is not None else 0, eps, freq.data_ptr() if n_rot else 0, n_rot, layout, amp, o_type,
          q_out.data_ptr() if q is not None else 0, ldo)
    return q_out


def window_workspace(cache: KVCache, window: Window, n_heads):
    """A workspace for moe_window_attention of n_heads heads (calls that overlap need one each)."""
    n = lib().moe_window_attention_bytes(cache.ref, window.ref, n_heads)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=cache.k.device)


def moe_window_attention(cache: KVCache, window: Window, q, scale, out=None, lse=None, ws=None, stream=None):
    """Attention of the window's queries (rows q [n_tokens, n_heads * head_dim]) over the cache, into out (rows like q,
    new if None), which is returned, and lse (float32 [n_tokens, n_heads], if given). ws: window_workspace's."""
    what = "moe_window_attention"
    if stream is not None:
        return _on_cache(stream, moe_window_attention, cache, window, q, scale, out, lse, ws)
    dev, n, d = _over_cache(what, cache, window), window.n_tokens, cache.head_dim
    ldq, size = _rows(what, "q", q, None, _HALVES, dev), q.shape
    wide = size[1]
    n_heads = wide // d
    if size[0] != n or wide % d:
        raise ValueError(f"{what}: q has shape {tuple(size)}, not {n} rows of heads of {d}")
    if out is None:
        out, ldo = q.new_empty((n, wide)), wide
    else:
        ldo = _rows(what, "out", out, size, (q.dtype,), dev)
    if lse is not None:
        _packed(what, "lse", lse, (n, n_heads), torch.float32, dev)
    if ws is None:
        ws = window_workspace(cache, window, n_heads)
    elif ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"{what}: ws is {ws.dtype} on {ws.device}, not contiguous bytes on the call's GPU")
    _call(what, dev, cache.ref, window.ref, _DTYPE[q.dtype], q.data_ptr(), ldq, n_heads, scale, out.data_ptr(), ldo,
          lse.data_ptr() if lse is not None else 0, ws.data_ptr(), ws.numel())
    return out


def logprobs_workspace(rows, n, k, device="cuda"):
    """A workspace for moe_token_logprobs (calls that overlap need one each)."""
    return torch.empty(max(lib().moe_token_logprobs_bytes(rows, n, k), 16), dtype=torch.uint8, device=device)


def moe_token_logprobs(logits, tokens=None, k=0, entropy=False, scale=1.0, ws=None, stream=None):
    """(logp, entropy, top_ids, top_logp) of logits rows [rows, n] under softmax(scale * logits): log probabilities float32
    [rows, given] of tokens (int32 [rows, given]), entropies [rows], and the k best tokens (int32 [rows, k]) with their log
    probabilities; None for what is not asked for. ws: logprobs_workspace's."""
    what = "moe_token_logprobs"
    if stream is not None:
        return _on(stream, moe_token_logprobs, logits, tokens, k, entropy, scale, ws)
    dev = _gpu(what, "logits", logits)
    ld = _rows(what, "logits", logits, None, _FLOATS, dev)
    rows, n = logits.shape
    given, logp, h, ids, top = 0, None, None, None, None
    if tokens is not None:
        if tokens.dim() != 2:
            raise ValueError(f"{what}: tokens has shape {tuple(tokens.shape)}, not rows")
        given = tokens.shape[1]
        _packed(what, "tokens", tokens, (rows, given), torch.int32, dev)
        logp = logits.new_empty((rows, given), dtype=torch.float32)
    if entropy:
        h = logits.new_empty((rows,), dtype=torch.float32)
    if not 0 <= k <= min(32, n) or given > 64:
        raise ValueError(f"{what}: {k} alternatives, {given} tokens a row, of {n}")
    if k:
        ids, top = logits.new_empty((rows, k), dtype=torch.int32), logits.new_empty((rows, k), dtype=torch.float32)
    if ws is None:
        ws = logprobs_workspace(rows, n, k, logits.device)
    elif ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"{what}: ws is {ws.dtype} on {ws.device}, not contiguous bytes on the call's GPU")
    _call(what, dev, _DTYPE[logits.dtype], logits.data_ptr(), ld, rows, n, scale, tokens.data_ptr() if given else 0, given,
          logp.data_ptr() if given else 0, h.data_ptr() if entropy else 0, k, ids.data_ptr() if k else 0,
          top.data_ptr() if k else 0, ws.data_ptr(), ws.numel())
    return logp, h, ids, top


# ------------------------------------------------------------------ bandwidth reference -------

def moe_stream_read(buf, out, grid, stream=None):
    """The achievable-bandwidth reference: one streaming read of `buf` (a contiguous device tensor
    of a multiple of 16 bytes) by `grid` workgroups; out[b] (uint32 or int32, >= grid words) gets
    the XOR of the 32-bit words workgroup b read."""
    assert buf.is_contiguous() and out.numel() >= grid and out.element_size() == 4
    _check(lib().moe_stream_read(_stream(stream), _ptr(buf), buf.numel() * buf.element_size(), _ptr(out),
                                 grid), "moe_stream_read")
