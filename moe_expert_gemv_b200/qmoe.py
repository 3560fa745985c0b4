"""Thin ctypes binding of libqmoe.so (C ABI in include/qmoe.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  Tensors are torch CUDA tensors (PyTorch supplies
device memory and the current stream); fp16 data travels as torch.float16,
packed words as torch.int32 (same bits as the uint32 words of the format).
A non-zero status raises QmoeError.  There is no CPU fallback: if the library
is missing or the device is not an sm_100 GPU the calls fail loudly.
"""
import ctypes
import functools
import os
import struct

import numpy as np
import torch

from . import build as _build

_lib = None

OK = 0
ERR_INVALID_ARG = -1
ERR_ALIGNMENT = -2
ERR_UNSUPPORTED = -3
ERR_CUDA = -4
ERR_DEVICE_STATUS = -5
ERR_TIMEOUT = -6
ERR_WORKSPACE = -7
DEV_BAD_EXPERT = 0x1
DEV_TIMEOUT = 0x2
DEV_BAD_PAGE = 0x4
DEV_BAD_TOKEN = 0x8


class QmoeError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__("%s: %s" % (what, status_string(code)))


class CQMatrix(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("biases", ctypes.c_void_p), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("group", ctypes.c_int32)]


class CMoeLayer(ctypes.Structure):
    _fields_ = [("gate", CQMatrix), ("up", CQMatrix), ("down", CQMatrix),
                ("sh_gate", CQMatrix), ("sh_up", CQMatrix), ("sh_down", CQMatrix),
                ("num_experts", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("inter", ctypes.c_int32)]


def lib():
    """Load libqmoe.so (building it first if it has never been built)."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not os.path.exists(path):
            _build.build()
        L = ctypes.CDLL(path)
        p, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        i64 = ctypes.c_int64
        sig = {
            "qgemv_affine": [p, p, i32, p, p, p],
            "qgemv_affine_workspace_bytes": [i32, i32, i32, i32],
            "qgemv_affine_ws": [p, p, i32, p, p, sz, p, p],
            "moe_expert_qmlp_ep": [p, p, p, p, i32, i32, i32, p, p, sz, p, p],
            "qmoe_f32_to_f16": [p, p, ctypes.c_int64, p],
            "qgemv_fmt": [p, p, i32, p, p, p],
            "qgemv_fmt_workspace_bytes": [i32, i32, i32, i32, i32],
            "qgemv_fmt_ws": [p, p, i32, p, p, sz, p, p],
            "moe_router_topk": [p, p, i32, i32, p, p, p, p, p],
            "moe_expert_workspace_bytes": [p, i32],
            "moe_expert_qmlp": [p, p, p, p, i32, p, p, sz, p, p],
            "moe_expert_gateup": [p, p, p, i32, p, sz, p, p],
            "moe_expert_down": [p, p, p, i32, p, p, sz, p, p],
            "moe_group_tokens": [p, i32, i32, i32, p, p, p, p, p],
            "moe_decode_pack_bytes": [p],
            "moe_decode_pack_layer": [p, p, p, sz, p],
            "moe_decode_workspace_bytes": [i32, i32, i32, i32],
            "moe_decode_layers": [p, i32, i32, i32, i32, p, i32, p, p, p, p, p, sz, p, p],
            "moe_decode_layers_host": [p, i32, i32, i32, i32, p, p, i32, p, p, p, sz, p, p],
            "moe_prefill_workspace_bytes": [p, i32, i32],
            "moe_prefill_qgemm": [p, p, i32, p, p, i32, p, p, sz, p, p],
            "rope_frequencies": [i32, ctypes.c_double, i32, ctypes.c_double, i32, ctypes.c_double,
                                 ctypes.c_double, p, p],
            "rope_rotate": [p, p, i64, i64, i32, i32, i32, i32, p, p, i64, i64, p, p],
            "kv_append": [p, p, p, p, p, p, i32, p, p, p, p],
            "attn_paged_workspace_bytes": [i32, i64],
            "attn_paged": [p, p, p, p, sz, p, p],
            "logits_process": [p, p, i64, i32, i32, i32, p, i64, p, sz, p, p],
            "logits_process_workspace_bytes": [i32, i32],
            "qmoe_pack_codes": [p, i32, i32, i32, p, p],
            "qmoe_unpack_codes": [p, i32, i32, i32, p, p],
            "qmoe_check_status": [p, p, p],
            "qmoe_status_string": [ctypes.c_int],
            "qmoe_set_dependent_launch": [i32],
            "qmoe_set_prefill_tensor_min": [i32],
            "qmoe_set_decode_wait_limit_ns": [ctypes.c_uint64],
            "qmoe_set_attn_wait_limit_ns": [ctypes.c_uint64],
            "qmoe_version": [],
            "qmoe_lfu_create": [i32, p],
            "qmoe_lfu_destroy": [p],
            "qmoe_lfu_plan": [p, p, i32, p, p, p],
            "qmoe_lfu_slots": [p, p, p],
            "qmoe_cache_create": [p, p, p],
            "qmoe_cache_destroy": [p],
            "moe_cache_layer": [p, p, p, i32, p, p, p, p, sz, p, p, p],
            "qmoe_cache_stats": [p, p, p, p, p],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.moe_expert_workspace_bytes.restype = sz
        L.qgemv_affine_workspace_bytes.restype = sz
        L.qgemv_fmt_workspace_bytes.restype = sz
        L.moe_prefill_workspace_bytes.restype = sz
        L.moe_decode_workspace_bytes.restype = sz
        L.moe_decode_pack_bytes.restype = sz
        L.attn_paged_workspace_bytes.restype = sz
        L.logits_process_workspace_bytes.restype = sz
        L.qmoe_status_string.restype = ctypes.c_char_p
        L.qmoe_version.restype = i32
        L.qmoe_set_dependent_launch.restype = i32
        L.qmoe_set_prefill_tensor_min.restype = i32
        L.qmoe_set_decode_wait_limit_ns.restype = ctypes.c_uint64
        L.qmoe_set_attn_wait_limit_ns.restype = ctypes.c_uint64
        L.qmoe_lfu_destroy.restype = None
        L.qmoe_cache_destroy.restype = None
        L.qmoe_lfu_plan.restype = i32
        _lib = L
    return _lib


def status_string(code):
    return lib().qmoe_status_string(int(code)).decode()


def _check(code, what):
    if code != OK:
        raise QmoeError(code, what)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(None)


def _need(t, dtype, what, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % what)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    return t


# ----------------------------------------------------------------- weights --
class QMatrix:
    """One affine-quantized matrix (or a stack of `stack` of them) on the GPU.

    packed: int32 [*, rows, cols*bits/32]; scales/biases: float16 [*, rows, cols/64]."""

    def __init__(self, packed, scales, biases, rows, cols, bits, stack=1):
        self.packed, self.scales, self.biases = packed, scales, biases
        self.rows, self.cols, self.bits, self.stack = rows, cols, bits, stack
        _need(packed, torch.int32, "packed")
        _need(scales, torch.float16, "scales")
        _need(biases, torch.float16, "biases")
        if packed.numel() != stack * rows * cols * bits // 32:
            raise ValueError("packed has %d words, expected %d" %
                             (packed.numel(), stack * rows * cols * bits // 32))
        if scales.numel() != stack * rows * cols // 64 or biases.numel() != scales.numel():
            raise ValueError("scales/biases size mismatch")
        self.c = CQMatrix(packed.data_ptr(), scales.data_ptr(), biases.data_ptr(), rows, cols,
                          bits, 64)

    @classmethod
    def from_numpy(cls, P, S, B, rows, cols, bits, device="cuda"):
        """From (packed uint32, scales/biases fp16 bits as uint16) numpy arrays."""
        stack = P.size // (rows * cols * bits // 32)
        packed = torch.from_numpy(P.view("int32").copy()).to(device)
        scales = torch.from_numpy(S.view("float16").copy()).to(device)
        biases = torch.from_numpy(B.view("float16").copy()).to(device)
        return cls(packed, scales, biases, rows, cols, bits, stack)


FMT_ZP4_BF16, FMT_SYM8_BF16 = 1, 2


class CQMatrixFmt(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("params", ctypes.c_void_p),
                ("rht_signs", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("cols", ctypes.c_int32), ("group", ctypes.c_int32), ("format", ctypes.c_int32)]


class QMatrixFmt:
    """A bf16-scale format-variant matrix on the GPU (zero-point 4-bit or
    symmetric 8-bit), optionally with the block-32 Hadamard rotation signs.

    packed: int32 [rows, cols*bits/32]; params: int32 [rows, cols/64];
    signs: int32 [cols/32] or None."""

    def __init__(self, packed, params, signs, rows, cols, fmt):
        if fmt not in (FMT_ZP4_BF16, FMT_SYM8_BF16):
            raise ValueError("unknown format %r" % (fmt,))
        bits = 4 if fmt == FMT_ZP4_BF16 else 8
        _need(packed, torch.int32, "packed", (rows, cols * bits // 32))
        _need(params, torch.int32, "params", (rows, cols // 64))
        if signs is not None:
            _need(signs, torch.int32, "signs", (cols // 32,))
        self.packed, self.params, self.signs = packed, params, signs
        self.rows, self.cols, self.fmt, self.bits = rows, cols, fmt, bits
        self.c = CQMatrixFmt(packed.data_ptr(), params.data_ptr(),
                             signs.data_ptr() if signs is not None else None, rows, cols, 64, fmt)

    @classmethod
    def from_numpy(cls, P, params, signs, rows, cols, fmt, rotate=True, device="cuda"):
        """From uint32 numpy arrays; `rotate` False drops the rotation."""
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.uint32).view("int32").copy()).to(device)
        return cls(t(P), t(params), t(signs) if rotate else None, rows, cols, fmt)


class MoELayer:
    """Routed experts (stacked gate/up/down) + shared expert (+ optional router)."""

    def __init__(self, gate, up, down, sh_gate, sh_up, sh_down, num_experts, hidden, inter,
                 router=None):
        self.mats = dict(gate=gate, up=up, down=down, sh_gate=sh_gate, sh_up=sh_up,
                         sh_down=sh_down)
        self.router = router
        self.num_experts, self.hidden, self.inter = num_experts, hidden, inter
        self.c = CMoeLayer(gate.c, up.c, down.c, sh_gate.c, sh_up.c, sh_down.c, num_experts,
                           hidden, inter)

    @classmethod
    def from_numpy(cls, m, E, H, I, device="cuda", rank=0, world=1):
        """From a dict like moe_expert_gemv_b200.synth.moe_layer() returns.
        With world > 1, the routed gate/up/down keep only the E/world experts
        rank `rank` holds (for moe_expert_qmlp_ep); shared expert and router
        are whole on every rank."""
        if E % world or not 0 <= rank < world:
            raise ValueError("world must divide E and 0 <= rank < world")
        lo, hi = rank * (E // world), (rank + 1) * (E // world)
        q = {}
        for name, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I),
                                 ("sh_gate", I, H), ("sh_up", I, H), ("sh_down", H, I)):
            arrs = m[name]
            if world > 1 and not name.startswith("sh_"):
                arrs = tuple(a[lo:hi] for a in arrs)
            q[name] = QMatrix.from_numpy(*arrs, rows, cols, 4, device)
        router = None
        if "router" in m:
            router = QMatrix.from_numpy(*m["router"], E, H, 8, device)
        return cls(q["gate"], q["up"], q["down"], q["sh_gate"], q["sh_up"], q["sh_down"], E, H,
                   I, router)


def expert_owner(e, E, world):
    """Rank that holds expert e when E experts are split over `world` ranks."""
    return e // (E // world)


def moe_expert_qmlp_ep(G, x, idx, weights, rank, world, y_partial=None, workspace=None,
                       status=None):
    """This rank's share of an expert-parallel MoE layer (G from
    MoELayer.from_numpy(..., rank=rank, world=world)): fp32 [H] partial,
    shared expert on rank 0.  The partials of all ranks sum to the layer
    output before its rounding to fp16."""
    x = _need(x, torch.float16, "x")
    top_k = idx.numel()
    if y_partial is None:
        y_partial = torch.empty(G.hidden, dtype=torch.float32, device=x.device)
    _need(y_partial, torch.float32, "y_partial", (G.hidden,))
    ws = workspace if workspace is not None else expert_workspace(G, top_k, x.device)
    _check(lib().moe_expert_qmlp_ep(ctypes.byref(G.c), _ptr(x), _ptr(idx), _ptr(weights), top_k,
                                    rank, world, _ptr(y_partial), _ptr(ws), ws.numel(), _ptr(status),
                                    _stream()), "moe_expert_qmlp_ep")
    return y_partial


def f32_to_f16(src, dst=None):
    """fp32 -> fp16 (round to nearest even) in the library's kernel."""
    src = _need(src, torch.float32, "src")
    if dst is None:
        dst = torch.empty(src.shape, dtype=torch.float16, device=src.device)
    _check(lib().qmoe_f32_to_f16(_ptr(src), _ptr(dst), src.numel(), _stream()), "qmoe_f32_to_f16")
    return dst


def moe_layer_ep(G, x, idx, weights, group=None, workspace=None):
    """One expert-parallel MoE layer on this rank of `group` (torch.distributed,
    NCCL on GPUs): the rank's partial, one all-reduce of the [H] fp32
    partials, then fp16.  Every rank passes the same x, idx and weights (the
    router is replicated)."""
    import torch.distributed as dist
    rank, world = dist.get_rank(group), dist.get_world_size(group)
    yp = moe_expert_qmlp_ep(G, x, idx, weights, rank, world, workspace=workspace)
    dist.all_reduce(yp, group=group)
    return f32_to_f16(yp)


# ------------------------------------------------------- expert streaming --
class LfuPlan:
    """The library's per-layer LFU expert-cache plan alone (host memory only,
    no GPU): step(ids) -> (slot_of [k], [(expert, slot), ...] misses)."""

    def __init__(self, nslots=16):
        h = ctypes.c_void_p()
        _check(lib().qmoe_lfu_create(nslots, ctypes.byref(h)), "qmoe_lfu_create")
        self.h, self.nslots = h, nslots

    def step(self, ids):
        ids = np.ascontiguousarray(ids, np.int32)
        k = ids.size
        slot_of = np.empty(max(k, 1), np.int32)
        me = np.empty(max(k, 1), np.int32)
        ms = np.empty(max(k, 1), np.int32)
        v = lambda a: a.ctypes.data_as(ctypes.c_void_p)
        n = lib().qmoe_lfu_plan(self.h, v(ids), k, v(slot_of), v(me), v(ms))
        if n < 0:
            raise ValueError("k > nslots, k > 16 or repeated ids")
        return slot_of[:k], list(zip(me[:n].tolist(), ms[:n].tolist()))

    def slots(self):
        e = np.empty(self.nslots, np.int32)
        c = np.empty(self.nslots, np.int64)
        _check(lib().qmoe_lfu_slots(self.h, e.ctypes.data_as(ctypes.c_void_p),
                                    c.ctypes.data_as(ctypes.c_void_p)), "qmoe_lfu_slots")
        return e, c

    def __del__(self):
        if getattr(self, "h", None) and _lib is not None:
            _lib.qmoe_lfu_destroy(self.h)
            self.h = None


class ExpertCacheLayer:
    """One MoE layer whose routed experts live in pinned host memory and are
    streamed into `nslots` device slots through the library's LFU plan; the
    router and the shared expert stay on the device."""

    def __init__(self, m, E, H, I, nslots=16, device="cuda"):
        self.E, self.H, self.I, self.nslots = E, H, I, nslots
        pin = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a).view(dt).copy()).pin_memory()
        self.host = {}
        for name in ("gate", "up", "down"):
            P, S, B = m[name]
            self.host[name] = (pin(P, np.int32), pin(S, np.float16), pin(B, np.float16))
        dims = {"gate": (I, H), "up": (I, H), "down": (H, I)}
        hq = {n: CQMatrix(t[0].data_ptr(), t[1].data_ptr(), t[2].data_ptr(), dims[n][0],
                          dims[n][1], 4, 64) for n, t in self.host.items()}
        dev_layer = MoELayer.from_numpy(m, E, H, I, device)   # router + shared expert on device
        self.router = dev_layer.router
        self.shared = {n: dev_layer.mats[n] for n in ("sh_gate", "sh_up", "sh_down")}
        self.slot = {}
        for n, (rows, cols) in dims.items():
            self.slot[n] = QMatrix(
                torch.zeros(nslots * rows * cols // 8, dtype=torch.int32, device=device),
                torch.zeros(nslots * rows * (cols // 64), dtype=torch.float16, device=device),
                torch.zeros(nslots * rows * (cols // 64), dtype=torch.float16, device=device),
                rows, cols, 4, nslots)
        sh = self.shared
        self.c_host = CMoeLayer(hq["gate"], hq["up"], hq["down"], sh["sh_gate"].c, sh["sh_up"].c,
                                sh["sh_down"].c, E, H, I)
        self.slot_layer = MoELayer(self.slot["gate"], self.slot["up"], self.slot["down"],
                                   sh["sh_gate"], sh["sh_up"], sh["sh_down"], nslots, H, I)
        h = ctypes.c_void_p()
        _check(lib().qmoe_cache_create(ctypes.byref(self.c_host), ctypes.byref(self.slot_layer.c),
                                       ctypes.byref(h)), "qmoe_cache_create")
        self.h = h
        self.workspace = {}
        self.copy_stream = torch.cuda.Stream(device=device)

    def forward(self, x, top_k=8, y=None, idx=None, weights=None, status=None):
        """One decode token x [H] float16 through the layer; returns y [H]."""
        x = _need(x, torch.float16, "x").reshape(-1)
        if y is None:
            y = torch.empty(self.H, dtype=torch.float16, device=x.device)
        ws = self.workspace.get(top_k)
        if ws is None:
            ws = self.workspace[top_k] = expert_workspace(self.slot_layer, top_k, x.device)
        _check(lib().moe_cache_layer(self.h, ctypes.byref(self.router.c), _ptr(x), top_k, _ptr(y),
                                     _ptr(idx), _ptr(weights), _ptr(ws), ws.numel(), _ptr(status),
                                     _stream(), ctypes.c_void_p(self.copy_stream.cuda_stream)),
               "moe_cache_layer")
        return y

    def stats(self):
        """(hits, misses, bytes copied, expert held by each slot)."""
        hits, misses, nbytes = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        slots = np.empty(self.nslots, np.int32)
        _check(lib().qmoe_cache_stats(self.h, ctypes.byref(hits), ctypes.byref(misses),
                                      ctypes.byref(nbytes),
                                      slots.ctypes.data_as(ctypes.c_void_p)), "qmoe_cache_stats")
        return hits.value, misses.value, nbytes.value, slots

    def __del__(self):
        if getattr(self, "h", None) and _lib is not None:
            _lib.qmoe_cache_destroy(self.h)
            self.h = None


# ------------------------------------------------------------- operations --
# zero-filled workspace of qgemv_affine_ws, one per device (allocated by the
# first call that needs it, so a CUDA graph captured after a first call
# reuses it); calls that can run at the same time on different streams must
# pass their own workspace
_qgemv_ws = {}


def qgemv_workspace(W, batch, device=None):
    """A zero-filled workspace for qgemv_affine_ws calls on W at this batch
    (None when none is needed)."""
    need = lib().qgemv_affine_workspace_bytes(W.rows, W.cols, W.bits, batch)
    if not need:
        return None
    return torch.zeros(need, dtype=torch.uint8, device=device or torch.device("cuda"))


def _shared_workspace(nbytes, device):
    ws = _qgemv_ws.get(device.index)
    if ws is None or ws.numel() < nbytes:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("qgemv_affine: no workspace of %d bytes yet on this device; call it "
                               "once before capturing, or pass workspace=" % nbytes)
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _qgemv_ws[device.index] = ws
    return ws


def qgemv_affine(W, x, y=None, status=None, one_pass=True, workspace=None):
    """y[b] = W x[b] for x [B][K] float16 (B <= 32).  Returns y [B][N] float16.
    A batch of 9..32 runs in one pass over the weights (qgemv_affine_ws) where
    the shape allows it, with `workspace` (a zero-filled uint8 tensor, see
    qgemv_workspace) or else one kept per device; one_pass=False runs one
    qGEMV launch per 8 rows (qgemv_affine)."""
    x = _need(x, torch.float16, "x")
    x2 = x.reshape(-1, W.cols)
    B = x2.shape[0]
    if y is None:
        y = torch.empty(B, W.rows, dtype=torch.float16, device=x.device)
    _need(y, torch.float16, "y", (B, W.rows))
    need = lib().qgemv_affine_workspace_bytes(W.rows, W.cols, W.bits, B) if one_pass and B > 8 else 0
    if need:
        ws = workspace if workspace is not None else _shared_workspace(need, x.device)
        _check(lib().qgemv_affine_ws(ctypes.byref(W.c), _ptr(x2), B, _ptr(y), _ptr(ws),
                                     ws.numel() * ws.element_size(), _ptr(status), _stream()),
               "qgemv_affine_ws")
    else:
        _check(lib().qgemv_affine(ctypes.byref(W.c), _ptr(x2), B, _ptr(y), _ptr(status),
                                  _stream()), "qgemv_affine")
    return y


def qgemv_fmt(W, x, y=None, status=None, one_pass=True, workspace=None):
    """y[b] = W (R x[b]) (R the rotation when W has signs) for x [B][K]
    float16 (B <= 32), W a QMatrixFmt.  Returns y [B][N] float16.  A batch
    of 9..32 runs in one pass over the weights (qgemv_fmt_ws) where the shape
    allows it (workspace as qgemv_affine); one_pass=False runs one launch per
    8 rows."""
    x = _need(x, torch.float16, "x")
    x2 = x.reshape(-1, W.cols)
    B = x2.shape[0]
    if y is None:
        y = torch.empty(B, W.rows, dtype=torch.float16, device=x.device)
    _need(y, torch.float16, "y", (B, W.rows))
    rotated = 1 if W.c.rht_signs else 0
    need = (lib().qgemv_fmt_workspace_bytes(W.rows, W.cols, W.c.format, rotated, B)
            if one_pass and B > 8 else 0)
    if one_pass and B > 8:
        ws = None
        if need:
            ws = workspace if workspace is not None else _shared_workspace(need, x.device)
        _check(lib().qgemv_fmt_ws(ctypes.byref(W.c), _ptr(x2), B, _ptr(y), _ptr(ws),
                                  0 if ws is None else ws.numel() * ws.element_size(),
                                  _ptr(status), _stream()), "qgemv_fmt_ws")
    else:
        _check(lib().qgemv_fmt(ctypes.byref(W.c), _ptr(x2), B, _ptr(y), _ptr(status), _stream()),
               "qgemv_fmt")
    return y


def moe_router_topk(router, x, top_k, idx=None, weights=None, logits=None, want_logits=False,
                    status=None):
    """Router logits -> softmax -> top-k -> renormalised weights for x [T][K].
    Returns (idx int32 [T][k], weights float32 [T][k], logits float32 [T][E] or None)."""
    x = _need(x, torch.float16, "x")
    x2 = x.reshape(-1, router.cols)
    T = x2.shape[0]
    dev = x.device
    if idx is None:
        idx = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(T, top_k, dtype=torch.float32, device=dev)
    if logits is None and want_logits:
        logits = torch.empty(T, router.rows, dtype=torch.float32, device=dev)
    _need(idx, torch.int32, "idx", (T, top_k))
    _need(weights, torch.float32, "weights", (T, top_k))
    if logits is not None:
        _need(logits, torch.float32, "logits", (T, router.rows))
    _check(lib().moe_router_topk(ctypes.byref(router.c), _ptr(x2), T, top_k, _ptr(idx),
                                 _ptr(weights), _ptr(logits), _ptr(status), _stream()),
           "moe_router_topk")
    return idx, weights, logits


def moe_expert_workspace_bytes(layer, top_k):
    return lib().moe_expert_workspace_bytes(ctypes.byref(layer.c), top_k)


def expert_workspace(layer, top_k, device="cuda"):
    """A zero-filled workspace for moe_expert_qmlp (reusable across calls)."""
    n = moe_expert_workspace_bytes(layer, top_k)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def moe_expert_qmlp(layer, x, idx, weights, y=None, workspace=None, status=None):
    """y = shared(x) + sum_j weights[j] * expert_{idx[j]}(x) for one token x [H]."""
    x = _need(x, torch.float16, "x").reshape(-1)
    top_k = idx.numel()
    _need(idx, torch.int32, "idx")
    _need(weights, torch.float32, "weights")
    if y is None:
        y = torch.empty(layer.hidden, dtype=torch.float16, device=x.device)
    if workspace is None:
        workspace = expert_workspace(layer, top_k, x.device)
    _check(lib().moe_expert_qmlp(ctypes.byref(layer.c), _ptr(x), _ptr(idx), _ptr(weights), top_k,
                                 _ptr(y), _ptr(workspace), workspace.numel(), _ptr(status),
                                 _stream()), "moe_expert_qmlp")
    return y


def moe_expert_gateup(layer, x, idx, workspace, status=None):
    x = _need(x, torch.float16, "x").reshape(-1)
    _check(lib().moe_expert_gateup(ctypes.byref(layer.c), _ptr(x), _ptr(idx), idx.numel(),
                                   _ptr(workspace), workspace.numel(), _ptr(status), _stream()),
           "moe_expert_gateup")


def moe_expert_down(layer, idx, weights, y, workspace, status=None):
    _check(lib().moe_expert_down(ctypes.byref(layer.c), _ptr(idx), _ptr(weights), idx.numel(),
                                 _ptr(y), _ptr(workspace), workspace.numel(), _ptr(status),
                                 _stream()), "moe_expert_down")
    return y


class DecodeStack:
    """A stack of MoE layers (each with its router) repacked once into the
    fused decode kernel's streaming layout, plus its zero-filled workspace."""

    def __init__(self, layers, top_k, device="cuda"):
        self.layers = list(layers)
        L0 = self.layers[0]
        self.top_k = top_k
        self.E, self.H, self.I = L0.num_experts, L0.hidden, L0.inter
        nbytes = lib().moe_decode_pack_bytes(ctypes.byref(L0.c))
        if nbytes == 0:
            raise ValueError("layer shape not supported by the fused decode")
        self.packed = []
        for L in self.layers:
            buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
            _check(lib().moe_decode_pack_layer(ctypes.byref(L.c), ctypes.byref(L.router.c),
                                               _ptr(buf), nbytes, _stream()),
                   "moe_decode_pack_layer")
            self.packed.append(buf)
        torch.cuda.current_stream().synchronize()
        self.c_packed = (ctypes.c_void_p * len(self.packed))(*[b.data_ptr() for b in self.packed])
        ws = lib().moe_decode_workspace_bytes(self.E, self.H, self.I, top_k)
        self.workspace = torch.zeros(ws, dtype=torch.uint8, device=device)


def moe_decode_layers(stack, x, y=None, idx=None, weights=None, logits=None, status=None):
    """One token per layer through the whole stack in one fused launch.
    x, y: float16 [n_layers][hidden]; idx int32 / weights float32 [n_layers][top_k];
    logits float32 [n_layers][num_experts] (optional)."""
    n = len(stack.packed)
    x = _need(x, torch.float16, "x", (n, stack.H))
    if y is None:
        y = torch.empty(n, stack.H, dtype=torch.float16, device=x.device)
    _need(y, torch.float16, "y", (n, stack.H))
    if idx is not None:
        _need(idx, torch.int32, "idx", (n, stack.top_k))
    if weights is not None:
        _need(weights, torch.float32, "weights", (n, stack.top_k))
    if logits is not None:
        _need(logits, torch.float32, "logits", (n, stack.E))
    _check(lib().moe_decode_layers(stack.c_packed, n, stack.E, stack.H, stack.I, _ptr(x),
                                   stack.top_k, _ptr(y), _ptr(idx), _ptr(weights), _ptr(logits),
                                   _ptr(stack.workspace), stack.workspace.numel(), _ptr(status),
                                   _stream()), "moe_decode_layers")
    return y


def moe_decode_layers_host(stack, x_host, y_host, x_dev, y_dev, status=None):
    """The decode step from host buffers through the C call that copies them:
    x_host -> x_dev, the fused decode, y_dev -> y_host, enqueued on the
    current stream (synchronise before reading y_host).  x_host / y_host:
    float16 [n_layers][hidden] CPU tensors (pinned for asynchronous copies);
    x_dev / y_dev: device staging tensors of the same shape."""
    n = len(stack.packed)
    for t, name in ((x_host, "x_host"), (y_host, "y_host")):
        if t.device.type != "cpu" or t.dtype != torch.float16 or tuple(t.shape) != (n, stack.H) \
                or not t.is_contiguous():
            raise ValueError("%s: expected a contiguous CPU float16 [%d, %d] tensor" % (name, n, stack.H))
    _need(x_dev, torch.float16, "x_dev", (n, stack.H))
    _need(y_dev, torch.float16, "y_dev", (n, stack.H))
    _check(lib().moe_decode_layers_host(stack.c_packed, n, stack.E, stack.H, stack.I,
                                        ctypes.c_void_p(x_host.data_ptr()),
                                        ctypes.c_void_p(y_host.data_ptr()), stack.top_k,
                                        _ptr(x_dev), _ptr(y_dev), _ptr(stack.workspace),
                                        stack.workspace.numel(), _ptr(status), _stream()),
           "moe_decode_layers_host")
    return y_host


def moe_group_tokens(idx, num_experts, status=None):
    """Counting sort of a chunk's (token, slot) pairs by expert.
    Returns (counts [E], offsets [E+1], pairs [T*k]) int32."""
    _need(idx, torch.int32, "idx")
    T, k = idx.shape
    dev = idx.device
    counts = torch.empty(num_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    pairs = torch.empty(T * k, dtype=torch.int32, device=dev)
    _check(lib().moe_group_tokens(_ptr(idx), T, k, num_experts, _ptr(counts), _ptr(offsets),
                                  _ptr(pairs), _ptr(status), _stream()), "moe_group_tokens")
    return counts, offsets, pairs


def moe_prefill_workspace_bytes(layer, tokens, top_k):
    return lib().moe_prefill_workspace_bytes(ctypes.byref(layer.c), tokens, top_k)


def moe_prefill_qgemm(layer, x, idx, weights, y=None, workspace=None, status=None):
    """y[t] = shared(x[t]) + sum_j weights[t][j] expert_{idx[t][j]}(x[t]), x [T][H]."""
    x = _need(x, torch.float16, "x")
    T = x.shape[0]
    _need(idx, torch.int32, "idx")
    _need(weights, torch.float32, "weights")
    top_k = idx.shape[1]
    if y is None:
        y = torch.empty(T, layer.hidden, dtype=torch.float16, device=x.device)
    if workspace is None:
        workspace = torch.empty(moe_prefill_workspace_bytes(layer, T, top_k), dtype=torch.uint8,
                                device=x.device)
    _check(lib().moe_prefill_qgemm(ctypes.byref(layer.c), _ptr(x), T, _ptr(idx), _ptr(weights),
                                   top_k, _ptr(y), _ptr(workspace), workspace.numel(),
                                   _ptr(status), _stream()), "moe_prefill_qgemm")
    return y


# ------------------------------------- positions, paged cache, attention --
class CKVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class CKVBatch(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("max_new", ctypes.c_int32)]


class CRope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("scale", ctypes.c_float)]


class CRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class CAttn(ctypes.Structure):
    _fields_ = [("q", CRows), ("out", CRows), ("lse", ctypes.c_void_p), ("heads", ctypes.c_int32),
                ("window", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float)]


class CLogitRules(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("history_len", ctypes.c_void_p),
                ("prompt_len", ctypes.c_void_p), ("history_stride", ctypes.c_int64),
                ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("mask_stride", ctypes.c_int64), ("max_history", ctypes.c_int32),
                ("max_bias", ctypes.c_int32)]


def _packer(cls):
    """pack(*values) -> bytes laid out as the structure (nested ones flat):
    built several times as fast as a ctypes structure, which shows in a decode
    step's calls."""
    code = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f"}
    flat = lambda c: "".join(code[t] if t in code else flat(t) for _, t in c._fields_)  # noqa: E731
    return struct.Struct("@" + flat(cls)).pack


_pack_rows, _pack_attn, _pack_rules = _packer(CRows), _packer(CAttn), _packer(CLogitRules)
_pack_batch = _packer(CKVBatch)
_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_KINDS = {"plain": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}


def _raw_stream(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def _capturing(device):
    """Whether the current stream of `device`, current or not, is being captured."""
    if device.index == torch._C._cuda_getDevice():
        return torch._C._cuda_isCurrentStreamCapturing()
    with torch.cuda.device(device):
        return torch._C._cuda_isCurrentStreamCapturing()


def _device_call(fn, what, device, *args):
    """fn(*args, current stream of `device`) with `device` current."""
    if device.index == torch._C._cuda_getDevice():
        code = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            code = fn(*args, _raw_stream(device))
    if code != OK:
        raise QmoeError(code, what)


def _on(device, t, what):
    if t.device != device:
        raise ValueError("%s is on %s, the other tensors on %s" % (what, t.device, device))
    return t


def _opt(t, dtype, what, shape, device):
    """Address of an optional contiguous tensor (None: 0)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError("%s must be a %s tensor" % (what, dtype))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous and have shape %s" % (what, tuple(shape)))
    if t.get_device() != device.index:
        _on(device, t, what)
    return t.data_ptr()


def _new_like(x):
    """A contiguous tensor of x's shape and type (torch.empty costs twice as much)."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _status(t, device):
    """Address of an optional status word."""
    return None if t is None else _opt(t, torch.int32, "status", t.shape, device)


def _rows(t, what, dtype, device, shape):
    """Address, token and head stride of a [tokens][heads][dim] tensor of any
    token and head strides."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != device.index:
        raise TypeError("%s must be a %s tensor on %s" % (what, dtype, device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    s0, s1, s2 = t.stride()
    if s2 != 1 and shape[2] > 1:
        raise ValueError("%s: the elements of a head must follow each other" % what)
    # the stride of a dimension of one element says nothing
    return t.data_ptr(), s0 if shape[0] > 1 else 0, s1 if shape[1] > 1 else 0


class KVCache:
    """One layer's paged K/V cache: k, v float16 or bfloat16 [num_pages]
    [page_size][kv_heads][head_dim], both with the same strides (a transposed
    view of [num_pages][kv_heads][page_size][head_dim] tensors is as good).
    Other tensors are another cache: k and v cannot be replaced."""

    def __init__(self, k, v):
        for t, what in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4:
                raise TypeError("%s must be a CUDA tensor [pages][page size][heads][dim]" % what)
            if t.dtype not in (torch.float16, torch.bfloat16):
                raise TypeError("%s must be float16 or bfloat16" % what)
        if k.dtype != v.dtype or k.shape != v.shape or k.stride() != v.stride() or k.device != v.device:
            raise ValueError("k and v must agree in type, shape, strides and device")
        if k.stride(3) != 1:
            raise ValueError("the elements of a head must follow each other")
        self._k, self._v, self.device, self.dtype = k, v, k.device, k.dtype
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        strides = [k.stride(i) if k.shape[i] > 1 else 0 for i in range(3)]
        self.c = CKVCache(k.data_ptr(), v.data_ptr(), *strides, *k.shape, _DTYPES[k.dtype])
        self._ref = ctypes.addressof(self.c)

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, dtype=torch.float16, device="cuda"):
        n = (num_pages, page_size, kv_heads, head_dim)
        return cls(torch.empty(n, dtype=dtype, device=device), torch.empty(n, dtype=dtype, device=device))


class KVBatch:
    """A step's sequences: page_table int32 [B][max_pages], q_start int32
    [B + 1] (sequence b's new tokens are rows q_start[b] .. q_start[b+1]),
    kv_len int32 [B] (cached tokens with the new ones).  max_new: an upper
    bound of the new tokens per sequence, which chooses the kernel (0: unknown;
    63 decode sequences then take 141 us instead of 108).  Each can be replaced
    between calls by another of the same batch and device."""

    def __init__(self, page_table, q_start, kv_len, max_new=0):
        _need(page_table, torch.int32, "page_table")
        if page_table.dim() != 2 or page_table.numel() == 0:
            raise ValueError("page_table must be [batch][pages], not empty")
        self.device, self._batch = page_table.device, page_table.shape[0]
        self._held = None   # (tokens, the C struct for steps of so many rows)
        self._page_table, self.q_start, self.kv_len, self.max_new = page_table, q_start, kv_len, max_new

    def _lens(self, t, what, n):
        _need(t, torch.int32, what, (n,))
        self._held = None
        return _on(self.device, t, what)

    @property
    def page_table(self):
        return self._page_table

    @page_table.setter
    def page_table(self, t):
        _need(t, torch.int32, "page_table")
        if t.dim() != 2 or t.shape[0] != self._batch or t.shape[1] == 0:
            raise ValueError("page_table must be [%d][pages]" % self._batch)
        self._page_table, self._held = _on(self.device, t, "page_table"), None

    @property
    def q_start(self):
        return self._q_start

    @q_start.setter
    def q_start(self, t):
        self._q_start = self._lens(t, "q_start", self._batch + 1)

    @property
    def kv_len(self):
        return self._kv_len

    @kv_len.setter
    def kv_len(self, t):
        self._kv_len = self._lens(t, "kv_len", self._batch)

    @property
    def max_new(self):
        return self._max_new

    @max_new.setter
    def max_new(self, n):
        self._max_new, self._held = int(n), None

    def _c(self, tokens):
        """(tokens, the C struct for steps of so many rows, its max_new)."""
        held = self._held
        if held is None or held[0] != tokens:
            held = self._held = (tokens, _pack_batch(
                self._page_table.data_ptr(), self._q_start.data_ptr(), self._kv_len.data_ptr(), self._batch,
                self._page_table.shape[1], tokens, self._max_new), self._max_new)
        return held


def rope_frequencies(rot_dim, base=10000.0, kind="plain", factor=1.0, trained=0, low=1.0, high=4.0):
    """(float64 [rot_dim / 2] CPU tensor of radians per position, scale)."""
    f = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float64)
    scale = ctypes.c_float()
    _check(lib().rope_frequencies(rot_dim, base, ROPE_KINDS[kind], factor, trained, low, high,
                                  f.data_ptr(), ctypes.addressof(scale)), "rope_frequencies")
    return f, scale.value


class Rope:
    """Rotary positions: inv_freq float64 [rot_dim / 2] on the GPU, layout
    "half" or "interleaved", scale of the turned part.  Another table is another
    Rope: inv_freq cannot be replaced."""

    def __init__(self, inv_freq, layout="half", scale=1.0):
        _need(inv_freq, torch.float64, "inv_freq")
        if inv_freq.dim() != 1 or inv_freq.numel() == 0:
            raise ValueError("inv_freq must be [rot_dim / 2]")
        self._inv_freq, self.device, self.rot_dim = inv_freq, inv_freq.device, 2 * inv_freq.numel()
        self.c = CRope(inv_freq.data_ptr(), self.rot_dim, ROPE_LAYOUTS[layout], scale)
        self._ref = ctypes.addressof(self.c)

    inv_freq = property(lambda self: self._inv_freq)

    @classmethod
    def make(cls, rot_dim, layout="half", device="cuda", **kw):
        """With the frequencies of rope_frequencies(rot_dim, **kw)."""
        f, scale = rope_frequencies(rot_dim, **kw)
        return cls(f.to(device), layout, scale)


def rope_rotate(rope, x, positions, out=None, status=None):
    """x [T][H][D] float16 or bfloat16 turned to `positions` int32 [T]."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3 or x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("x must be a float16 or bfloat16 tensor [tokens][heads][dim]")
    dev = _on(rope.device, x, "x").device
    if out is None:
        out = _new_like(x)
    x_ptr, x_token, x_head = _rows(x, "x", x.dtype, dev, x.shape)
    o_ptr, o_token, o_head = _rows(out, "out", x.dtype, dev, x.shape)
    T, H, D = x.shape
    if x.numel() == 0:   # empty tensors have no address
        return out
    _device_call(lib().rope_rotate, "rope_rotate", dev, rope._ref, x_ptr, x_token, x_head, _DTYPES[x.dtype],
                 T, H, D, _opt(positions, torch.int32, "positions", (T,), dev), o_ptr, o_token, o_head,
                 _status(status, dev))
    return out


def kv_append(cache, batch, k, v, q=None, rope=None, positions=None, q_out=None, status=None):
    """Store a step's keys (turned by `rope`) and values [T][kv_heads][D] in
    the cache and return the step's queries q [T][heads][D] turned likewise
    (None without q), in one launch.  positions int32 [T]: the rotation's
    positions where they are not the rows' places in their sequences."""
    dev, dt = cache.device, cache.dtype
    if batch.device != dev or (rope is not None and rope.device != dev):
        raise ValueError("cache, batch and rope must be on one device")
    T = k.shape[0]
    shape = (T, cache.kv_heads, cache.head_dim)
    ck, cv = _pack_rows(*_rows(k, "k", dt, dev, shape)), _pack_rows(*_rows(v, "v", dt, dev, shape))
    cq = co = None
    heads = 0
    if q is not None:
        if rope is None:
            raise ValueError("q needs rope")
        heads = q.shape[1]
        shape = (T, heads, cache.head_dim)
        cq = _pack_rows(*_rows(q, "q", dt, dev, shape))
        if q_out is None:
            q_out = _new_like(q)
        co = _pack_rows(*_rows(q_out, "q_out", dt, dev, shape))
    if T == 0:   # empty tensors have no address
        return q_out
    _device_call(lib().kv_append, "kv_append", dev, cache._ref, batch._c(T)[1], rope._ref if rope else None,
                 _opt(positions, torch.int32, "positions", (T,), dev), cq, co, heads, ck, cv, _status(status, dev))
    return q_out


_ATTN_COUNTER_BYTES = 4096   # the part of a workspace that has to start as zeros
_attn_ws = {}


def attn_workspace(head_dim, max_rows, device="cuda"):
    """A workspace for attn_paged calls of at most max_rows = new tokens x
    query heads per K/V head rows in a sequence."""
    need = lib().attn_paged_workspace_bytes(head_dim, max_rows)
    if not need:
        raise ValueError("unsupported head_dim %d" % head_dim)
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    ws[:_ATTN_COUNTER_BYTES].zero_()
    return ws


@functools.lru_cache(maxsize=64)
def _attn_need(head_dim, max_rows):
    return lib().attn_paged_workspace_bytes(head_dim, max_rows)


def _attn_workspace(head_dim, max_rows, device):
    """One workspace for each stream; in a capture one of the graph's own (its
    zeros are set by the graph)."""
    if _capturing(device):
        return attn_workspace(head_dim, max_rows, device)
    key = (device.index, _raw_stream(device))
    ws = _attn_ws.get(key)
    if ws is None or ws.numel() < _attn_need(head_dim, max_rows):
        ws = _attn_ws[key] = attn_workspace(head_dim, max_rows, device)
    return ws


def attn_paged(cache, batch, q, out=None, lse=None, want_lse=False, scale=None, softcap=0.0, window=0,
               causal=True, workspace=None, status=None):
    """Attention of the step's queries q [T][heads][D] over the cache, which
    already holds the step's own keys and values.  scale: 1/sqrt(D) unless
    given; softcap > 0 caps the scores by a tanh; window > 0: a sliding window
    of that many keys.  Returns out [T][heads][D], or (out, lse float32
    [T][heads]) with want_lse or lse."""
    dev = cache.device
    if batch.device != dev:
        raise ValueError("cache and batch must be on one device")
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q must be a tensor [tokens][heads][dim]")
    T, H, D = q.shape
    shape = (T, H, cache.head_dim)
    q_ptr, q_token, q_head = _rows(q, "q", cache.dtype, dev, shape)
    if out is None:
        out = _new_like(q)
        o_ptr, o_token, o_head = out.data_ptr(), H * D, D
    else:
        o_ptr, o_token, o_head = _rows(out, "out", cache.dtype, dev, shape)
    if lse is None and want_lse:
        lse = torch.empty(T, H, dtype=torch.float32, device=dev)
    if T == 0:   # empty tensors have no address
        return out if lse is None else (out, lse)
    held = batch._c(T)
    if workspace is None:
        workspace = _attn_workspace(D, max((held[2] or T) * (H // cache.kv_heads), 1), dev)
    else:
        _on(dev, workspace, "workspace")
    c = _pack_attn(q_ptr, q_token, q_head, o_ptr, o_token, o_head,
                   0 if lse is None else _opt(lse, torch.float32, "lse", (T, H), dev), H, window, 1 if causal else 0,
                   D ** -0.5 if scale is None else scale, softcap)
    _device_call(lib().attn_paged, "attn_paged", dev, c, cache._ref, held[1], workspace.data_ptr(),
                 workspace.numel() * workspace.element_size(), None if status is None else _status(status, dev))
    return out if lse is None else (out, lse)


# --------------------------------------------------------- rules on logits --
_logits_ws = {}   # one workspace for each device and stream


@functools.lru_cache(maxsize=64)   # a history that grows is another width at every step
def _logits_need(rows, max_history):
    return lib().logits_process_workspace_bytes(rows, max_history)


def logits_process(logits, out=None, history=None, history_len=None, prompt_len=None, repetition=None,
                   presence=None, frequency=None, bias_ids=None, bias=None, mask=None, workspace=None, status=None):
    """Penalties, biases and a grammar mask on logits [rows][vocab] (float16,
    bfloat16 or float32); out may be logits itself.  history int32 [rows][n]
    with history_len int32 [rows] tokens in use, prompt_len of them the prompt;
    repetition, presence, frequency float32 [rows]; bias_ids int32 / bias
    float32 [rows][m] (-1: unused); mask int32 [rows] or [1] x [ceil(vocab /
    32)], bit v % 32 of word v / 32 set where token v is allowed."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dim() != 2 or logits.dtype not in _DTYPES:
        raise TypeError("logits must be a CUDA tensor [rows][vocab] of float16, bfloat16 or float32")
    R, V = logits.shape
    dev = logits.device
    in_stride, step = logits.stride()
    if out is None:
        out, out_stride = _new_like(logits), V
    else:
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError("out must be like logits")
        out_stride, out_step = _on(dev, out, "out").stride()
        step = 1 if step == out_step == 1 else 0
    if V > 1 and step != 1:
        raise ValueError("a row's logits must follow each other")
    hist = hist_stride = max_hist = mask_ptr = mask_stride = max_bias = 0
    if history is not None:
        if history.dim() != 2 or history.shape[0] != R or history.dtype != torch.int32 or \
                (history.shape[1] > 1 and history.stride(1) != 1):
            raise ValueError("history must be int32 [rows][tokens], the tokens of a row one after the other")
        if history_len is None:
            raise ValueError("history needs history_len")
        max_hist = history.shape[1]
        hist, hist_stride = _on(dev, history, "history").data_ptr(), history.stride(0) if R > 1 else max_hist
        if max_hist == 0:   # nothing written yet (and an empty tensor has no address): no penalties
            history_len = prompt_len = repetition = presence = frequency = None
            hist = hist_stride = 0
    elif any(t is not None for t in (history_len, prompt_len, repetition, presence, frequency)):
        raise ValueError("penalties need history")
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias and bias_ids go together")
    if bias is not None:
        max_bias = bias.shape[-1]
    if mask is not None:
        _need(mask, torch.int32, "mask")
        words = (V + 31) // 32
        if mask.dim() != 2 or mask.shape[0] not in (1, R) or mask.shape[1] < words:
            raise ValueError("mask must be int32 [rows] or [1] x at least %d words" % words)
        mask_ptr = _on(dev, mask, "mask").data_ptr()
        mask_stride = mask.shape[1] if mask.shape[0] == R else 0
    rows = (R,)
    c = _pack_rules(hist, _opt(history_len, torch.int32, "history_len", rows, dev),
                    _opt(prompt_len, torch.int32, "prompt_len", rows, dev), hist_stride,
                    _opt(repetition, torch.float32, "repetition", rows, dev),
                    _opt(presence, torch.float32, "presence", rows, dev),
                    _opt(frequency, torch.float32, "frequency", rows, dev),
                    _opt(bias_ids, torch.int32, "bias_ids", (R, max_bias), dev),
                    _opt(bias, torch.float32, "bias", (R, max_bias), dev), mask_ptr, mask_stride, max_hist, max_bias)
    if R == 0 or V == 0:   # empty tensors have no address
        return out
    ws = nbytes = 0
    need = _logits_need(R, max_hist)
    if workspace is not None:
        ws, nbytes = _on(dev, workspace, "workspace").data_ptr(), workspace.numel() * workspace.element_size()
    elif need:
        key = (dev.index, _raw_stream(dev))
        capturing = _capturing(dev)   # a capture's stays with its graph
        held = None if capturing else _logits_ws.get(key)
        if held is None or held.numel() < need:
            # room for a history that grows by a quarter
            held = torch.empty(need if capturing else need + need // 4, dtype=torch.uint8, device=dev)
            if not capturing:
                _logits_ws[key] = held
        ws, nbytes = held.data_ptr(), held.numel()
    _device_call(lib().logits_process, "logits_process", dev, c, logits.data_ptr(), in_stride if R > 1 else V,
                 _DTYPES[logits.dtype], R, V, out.data_ptr(), out_stride if R > 1 else V, ws, nbytes,
                 _status(status, dev))
    return out


def qmoe_pack_codes(codes, bits):
    """uint8 codes [rows][cols] -> int32 packed words [rows][cols*bits/32]."""
    _need(codes, torch.uint8, "codes")
    rows, cols = codes.shape
    packed = torch.empty(rows, cols * bits // 32, dtype=torch.int32, device=codes.device)
    _check(lib().qmoe_pack_codes(_ptr(codes), rows, cols, bits, _ptr(packed), _stream()),
           "qmoe_pack_codes")
    return packed


def qmoe_unpack_codes(packed, rows, cols, bits):
    _need(packed, torch.int32, "packed")
    codes = torch.empty(rows, cols, dtype=torch.uint8, device=packed.device)
    _check(lib().qmoe_unpack_codes(_ptr(packed), rows, cols, bits, _ptr(codes), _stream()),
           "qmoe_unpack_codes")
    return codes


def qmoe_check_status(status=None):
    """Synchronise the current stream; return the device flags (and clear them).
    Raises QmoeError on a CUDA failure; flags are returned, not raised."""
    flags = ctypes.c_int32(0)
    rc = lib().qmoe_check_status(_ptr(status), _stream(), ctypes.byref(flags))
    if rc not in (OK, -5, -6):
        raise QmoeError(rc, "qmoe_check_status")
    return flags.value


def qmoe_set_dependent_launch(enable):
    return bool(lib().qmoe_set_dependent_launch(1 if enable else 0))


def qmoe_set_decode_wait_limit_ns(ns):
    """Limit of every wait inside the fused decode (0: the default 2 s).
    Returns the previous setting."""
    return int(lib().qmoe_set_decode_wait_limit_ns(int(ns)))


def qmoe_set_attn_wait_limit_ns(ns):
    """Limit of every wait inside attn_paged (0: the default 2 s).  Returns the
    previous setting."""
    return int(lib().qmoe_set_attn_wait_limit_ns(int(ns)))


# the threshold used when the tensor-core prefill path is switched on (the
# library's own default is 0: off)
TENSOR_MIN_DEFAULT = 16


def qmoe_set_prefill_tensor_min(min_tokens):
    """Experts of a prefill chunk with at least min_tokens tokens run on the
    tensor-core kernels (0: none).  Returns the previous setting."""
    return int(lib().qmoe_set_prefill_tensor_min(int(min_tokens)))


def qmoe_version():
    return lib().qmoe_version()
