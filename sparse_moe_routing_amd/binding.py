"""ctypes binding of libmoe.so (include/moe.h): argument marshalling only.

Every step of the layer runs in the HIP kernels of libmoe.so; this module converts torch device
tensors to raw pointers and the current torch stream to a hipStream_t. PyTorch supplies device
memory (weights, activations, outputs, workspace) and streams, nothing else. If the library is
missing, loading raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_HIP = -4
MOE_F32 = 0
MOE_BF16 = 1
MOE_FP8_E4M3 = 2  # bf16 x and router; FP8 E4M3 expert weights with fp32 per-row scales
MOE_MXFP4 = 3  # bf16 x and router; MXFP4 expert weights (packed E2M1 codes, E8M0 bytes per 32)
DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8": MOE_FP8_E4M3, "mxfp4": MOE_MXFP4}
WEIGHT_KEYS = ("router_w", "router_bias", "gate_up", "down", "shared_gate_up", "shared_down",
               "gate_up_scale", "down_scale", "shared_gate_up_scale", "shared_down_scale")

EXPORTS = ("moe_create", "moe_destroy", "moe_workspace_bytes", "moe_workspace_state_bytes",
           "moe_route", "moe_bucket", "moe_bucket_rows",
           "moe_forward", "moe_forward_noalloc", "moe_forward_plan", "moe_forward_timed",
           "moe_permute", "moe_permute_backward", "moe_unpermute", "moe_unpermute_backward",
           "moe_quantize_i8", "moe_permute_i8", "moe_matmul_i8",
           "moe_status_str")


class moe_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("shared_inter", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class moe_weights(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in WEIGHT_KEYS]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe.so and declare its signatures. Raises if it has not been built."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m sparse_moe_routing_amd.build`"
                           " (there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.moe_create.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(moe_weights),
                               ctypes.POINTER(ctypes.c_void_p)]
    lib.moe_create.restype = ctypes.c_int
    lib.moe_destroy.argtypes = [P]
    lib.moe_destroy.restype = None
    lib.moe_workspace_bytes.argtypes = [P, I32]
    lib.moe_workspace_bytes.restype = SZ
    lib.moe_workspace_state_bytes.argtypes = [P]
    lib.moe_workspace_state_bytes.restype = SZ
    lib.moe_route.argtypes = [P, P, P, I32, P, P, P, P, P, SZ, P]
    lib.moe_route.restype = ctypes.c_int
    lib.moe_bucket.argtypes = [P, P, I32, P, P, P, P, SZ, P]
    lib.moe_bucket.restype = ctypes.c_int
    lib.moe_bucket_rows.argtypes = [P, P, I32, P, P, P, P, P, SZ, P]
    lib.moe_bucket_rows.restype = ctypes.c_int
    lib.moe_permute.argtypes = [P, P, I32, I32, I32, I32, P, P]
    lib.moe_permute.restype = ctypes.c_int
    lib.moe_permute_backward.argtypes = [P, P, I32, I32, I32, I32, P, P]
    lib.moe_permute_backward.restype = ctypes.c_int
    lib.moe_unpermute.argtypes = [P, P, P, P, P, I32, I32, I32, I32, P, I32, P]
    lib.moe_unpermute.restype = ctypes.c_int
    lib.moe_unpermute_backward.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, P, P, P, P, P]
    lib.moe_unpermute_backward.restype = ctypes.c_int
    lib.moe_quantize_i8.argtypes = [P, I32, I32, I32, P, P, P]
    lib.moe_quantize_i8.restype = ctypes.c_int
    lib.moe_permute_i8.argtypes = [P, P, I32, I32, I32, I32, P, P, P]
    lib.moe_permute_i8.restype = ctypes.c_int
    lib.moe_matmul_i8.argtypes = [P, P, I32, P, P, I32, I32, I32, P, I32, P, I32, P]
    lib.moe_matmul_i8.restype = ctypes.c_int
    lib.moe_forward.argtypes = [P, P, I32, P, P, P, P, P, SZ, P]
    lib.moe_forward.restype = ctypes.c_int
    lib.moe_forward_noalloc.argtypes = [P, P, I32, P, P, P, P, P]
    lib.moe_forward_noalloc.restype = ctypes.c_int
    lib.moe_forward_plan.argtypes = [P, I32, I32, ctypes.POINTER(I32),
                                     ctypes.POINTER(ctypes.c_char_p), I32]
    lib.moe_forward_plan.restype = ctypes.c_int
    lib.moe_forward_timed.argtypes = [P, P, I32, P, P, P, P, P, SZ, P, P, I32]
    lib.moe_forward_timed.restype = ctypes.c_int
    lib.moe_status_str.argtypes = [ctypes.c_int]
    lib.moe_status_str.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = load().moe_status_str(status).decode()
        super().__init__(f"{what}: {msg} ({status})")


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class MoeLayer:
    """A context over device weight tensors (borrowed: the tensors are kept alive here).

    weights: dict with router_w [R][H], router_bias [R] fp32 or None, gate_up [E][2I][H],
    down [E][H][I], shared_gate_up [2Is][H] or None, shared_down [H][Is] or None, and for "fp8"
    the row scales gate_up_scale [E][2I], down_scale [E][H], shared_gate_up_scale [2Is] and
    shared_down_scale [H] (fp32) next to uint8 FP8 E4M3 codes, for "mxfp4" packed E2M1 codes
    ([E][2I][H/2] ...) with E8M0 scale bytes gate_up_scale [E][2I][H/32], down_scale
    [E][H][I/32], shared_gate_up_scale [2Is][H/32], shared_down_scale [H][Is/32]; bf16 weights
    may be torch.bfloat16 or 16-bit integer tensors holding the bf16 bits.
    """

    def __init__(self, hidden, num_experts, inter, shared_inter, max_tokens, dtype, weights,
                 top_k=8):
        self.lib = load()
        self.cfg = moe_config(hidden, num_experts, top_k, inter, shared_inter, max_tokens,
                              DTYPES[dtype])
        self._keep = dict(weights)
        w = moe_weights(*((None if weights.get(k) is None else weights[k].data_ptr())
                          for k in WEIGHT_KEYS))
        ctx = ctypes.c_void_p()
        _check(self.lib.moe_create(ctypes.byref(self.cfg), ctypes.byref(w), ctypes.byref(ctx)),
               "moe_create")
        self.ctx = ctx
        self.hidden, self.num_experts = hidden, num_experts
        self.shared_inter = shared_inter
        self.rows = num_experts + (1 if shared_inter > 0 else 0)

    def close(self):
        if getattr(self, "ctx", None):
            self.lib.moe_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_bytes(self, T: int) -> int:
        return int(self.lib.moe_workspace_bytes(self.ctx, T))

    def state_bytes(self) -> int:
        """Size of the workspace's leading state region (zero before the first call, left zero
        by every call)."""
        return int(self.lib.moe_workspace_state_bytes(self.ctx))

    def workspace(self, T: int, device="cuda"):
        """A workspace for calls of up to T tokens. It starts zeroed: the library keeps arrival
        counters and work-queue words in its leading state region, which must be zero before the
        first call and which every call leaves at zero."""
        import torch
        return torch.zeros(max(self.workspace_bytes(T), 256), dtype=torch.uint8, device=device)

    def _zeroed(self, T, device, stream):
        """A workspace of one call: allocated for and zeroed on the stream that the call runs on
        (zeroed on another one it could still hold old counters when the kernels start, and be
        given away while they run)."""
        import torch
        with torch.cuda.stream(stream):
            return self.workspace(T, device)

    def route(self, x=None, logits=None, T=None, ws=None, want_logits=True, stream=None):
        """(logits [T][R] or None, ids [T][8], w [T][8], g [T] or None) from x or given logits."""
        import torch
        src = x if x is not None else logits
        T = src.shape[0] if T is None else T
        dev = src.device
        ids = torch.empty((T, 8), dtype=torch.int32, device=dev)
        w = torch.empty((T, 8), dtype=torch.float32, device=dev)
        g = torch.empty((T,), dtype=torch.float32, device=dev) if self.shared_inter > 0 else None
        z = torch.empty((T, self.rows), dtype=torch.float32, device=dev) if want_logits else None
        ws = self._zeroed(T, dev, stream) if ws is None else ws
        _check(self.lib.moe_route(self.ctx, _ptr(x), _ptr(logits), T, _ptr(z), _ptr(ids),
                                  _ptr(w), _ptr(g), _ptr(ws), ws.numel(), _stream(stream)),
               "moe_route")
        return z, ids, w, g

    def bucket(self, ids, ws=None, stream=None):
        """(counts [E], offsets [E+1], perm [T*8]) for ids [T][8]."""
        import torch
        T = ids.shape[0]
        dev = ids.device
        counts = torch.empty((self.num_experts,), dtype=torch.int32, device=dev)
        offsets = torch.empty((self.num_experts + 1,), dtype=torch.int32, device=dev)
        perm = torch.empty((T * 8,), dtype=torch.int32, device=dev)
        ws = self._zeroed(T, dev, stream) if ws is None else ws
        _check(self.lib.moe_bucket(self.ctx, _ptr(ids), T, _ptr(counts), _ptr(offsets),
                                   _ptr(perm), _ptr(ws), ws.numel(), _stream(stream)),
               "moe_bucket")
        return counts, offsets, perm

    def bucket_rows(self, ids, ws=None, stream=None):
        """(counts [E], offsets [E+1], perm [T*8], rows [T*8]): bucket() and the inverse of perm,
        the table that the row operators below take (-1: the pair's id is outside [0, E)). ids,
        device and stream are checked and used as by those operators."""
        import torch
        dev = ids.device
        ctx = _switched(dev, stream)
        if ctx is not None:
            with ctx:
                return self.bucket_rows(ids, ws)
        T = ids.shape[0]
        at = _want("ids", ids, torch.int32, (T, 8), dev.index)
        counts = torch.empty((self.num_experts,), dtype=torch.int32, device=dev)
        offsets = torch.empty((self.num_experts + 1,), dtype=torch.int32, device=dev)
        perm = torch.empty((T * 8,), dtype=torch.int32, device=dev)
        rows = torch.empty((T * 8,), dtype=torch.int32, device=dev)
        if T == 0:  # the library enqueues nothing: no pairs
            counts.zero_()
            offsets.zero_()
        ws = self.workspace(T, dev) if ws is None else ws
        _check(self.lib.moe_bucket_rows(self.ctx, at, T, _ptr(counts), _ptr(offsets), _ptr(perm),
                                        _ptr(rows), _ptr(ws), ws.numel(), _stream()),
               "moe_bucket_rows")
        return counts, offsets, perm, rows

    def forward(self, x, routing=None, y=None, ws=None, stream=None, events=None):
        """y [T][H] fp32; routing = (ids, w, g) to use a given routing, else routed from x."""
        import torch
        T = x.shape[0]
        dev = x.device
        y = torch.empty((T, self.hidden), dtype=torch.float32, device=dev) if y is None else y
        ws = self._zeroed(T, dev, stream) if ws is None else ws
        ids = w = g = None
        if routing is not None:
            ids, w, g = routing
        if events is None:
            _check(self.lib.moe_forward(self.ctx, _ptr(x), T, _ptr(ids), _ptr(w), _ptr(g),
                                        _ptr(y), _ptr(ws), ws.numel(), _stream(stream)),
                   "moe_forward")
        else:
            arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
            _check(self.lib.moe_forward_timed(self.ctx, _ptr(x), T, _ptr(ids), _ptr(w), _ptr(g),
                                              _ptr(y), _ptr(ws), ws.numel(), _stream(stream),
                                              arr, len(events)), "moe_forward_timed")
        return y

    def forward_noalloc(self, x, routing=None, y=None, stream=None):
        """moe_forward_noalloc: as forward, with the library's static scratch as workspace."""
        import torch
        T = x.shape[0]
        y = torch.empty((T, self.hidden), dtype=torch.float32, device=x.device) if y is None else y
        ids = w = g = None
        if routing is not None:
            ids, w, g = routing
        _check(self.lib.moe_forward_noalloc(self.ctx, _ptr(x), T, _ptr(ids), _ptr(w), _ptr(g),
                                            _ptr(y), _stream(stream)), "moe_forward_noalloc")
        return y

    def plan(self, T: int, routing_given: bool = False):
        """Names of the kernels moe_forward enqueues for T tokens, in order."""
        n = ctypes.c_int32()
        names = (ctypes.c_char_p * 16)()
        _check(self.lib.moe_forward_plan(self.ctx, T, int(routing_given), ctypes.byref(n), names,
                                         16), "moe_forward_plan")
        return [names[i].decode() for i in range(n.value)]


# ---------------------------------------------------------------- separate operators
# Rows sorted by expert and back, their gradients, and products of 8-bit integers, around a
# caller's own expert products. rows is the [T*8] int32 table of MoeLayer.bucket_rows. Tensors are
# contiguous and on one device; what is not raises ValueError before anything is enqueued, and a
# call that the library refuses raises MoeError. Without `stream` the work is enqueued on the
# current stream of the tensors' device; with it, results are allocated for that stream, and the
# caller orders it after whatever writes the inputs and keeps them until the work has run. A decode
# round's operators take a few microseconds each, so this side is kept short: no Stream object
# (three microseconds) is made where nothing has to be switched. permute and unpermute are recorded by
# autograd (autograd.py); the others give results without a gradient: 8-bit codes have none, and the
# gradients' own operators are not differentiated again.
_row_types = {}  # torch dtype -> the library's number (filled on first use)


def _want(name, t, dtype, shape, index):
    """Address of t, a contiguous tensor of the dtype and shape on GPU `index`."""
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _row_enum(name, dtype):
    """The library's number of a row type."""
    if not _row_types:
        import torch
        _row_types.update({torch.float32: MOE_F32, torch.bfloat16: MOE_BF16})
    num = _row_types.get(dtype)
    if num is None:
        raise ValueError(f"{name}: dtype {dtype}, expected torch.float32 or torch.bfloat16")
    return num


def _switched(device, stream):
    """Context in which the tensors' device is current and, if given, the stream on it; None when
    that is already so (and no stream is given)."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not on {device}")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream of {stream.device}, tensors on {device}")
        return torch.cuda.stream(stream)
    if device.index != torch._C._cuda_getDevice():
        return torch.cuda.device(device)
    return None


def _recorded(out, name):
    """For a call whose operands require a gradient: whether one is recorded. A result buffer given
    by the caller is refused then, as by torch's own operators."""
    import torch
    if not torch.is_grad_enabled():
        return False
    if out is not None:
        raise ValueError(f"{name} cannot be given where a gradient is recorded (use torch.no_grad())")
    return True


def permute(x, rows, n_rows=None, xs=None, stream=None):
    """xs [n_rows][H] with xs[rows[8t + k]] = x[t] for x [T][H] (fp32 or bf16); n_rows: by default
    T * 8, or the rows of xs. Rows that no pair names keep what xs held. Differentiable in x."""
    import torch
    dev = x.device
    ctx = _switched(dev, stream)
    if ctx is not None:
        with ctx:
            return permute(x, rows, n_rows, xs)
    if x.requires_grad and _recorded(xs, "xs"):
        from .autograd import Permute
        return Permute.apply(x, rows, n_rows)
    (T, H), dt, at = x.shape, x.dtype, dev.index
    num = _row_enum("x", dt)
    px, pr = _want("x", x, dt, (T, H), at), _want("rows", rows, torch.int32, (T * 8,), at)
    if xs is None:
        xs = torch.empty((T * 8 if n_rows is None else n_rows, H), dtype=dt, device=dev)
    n = xs.shape[0] if n_rows is None else n_rows
    _check(load().moe_permute(px, pr, T, H, n, num, _want("xs", xs, dt, (n, H), at),
                              torch._C._cuda_getCurrentRawStream(at)), "moe_permute")
    return xs


def permute_backward(dxs, rows, dx=None, stream=None):
    """dx [T][H] with dx[t] = sum_k dxs[rows[8t + k]]: the gradient of permute."""
    import torch
    dev = dxs.device
    ctx = _switched(dev, stream)
    if ctx is not None:
        with ctx:
            return permute_backward(dxs, rows, dx)
    (n, H), dt, at = dxs.shape, dxs.dtype, dev.index
    T = rows.numel() // 8
    num = _row_enum("dxs", dt)
    pd, pr = _want("dxs", dxs, dt, (n, H), at), _want("rows", rows, torch.int32, (T * 8,), at)
    if dx is None:
        dx = torch.empty((T, H), dtype=dt, device=dev)
    _check(load().moe_permute_backward(pd, pr, T, H, n, num, _want("dx", dx, dt, (T, H), at),
                                       torch._C._cuda_getCurrentRawStream(at)),
           "moe_permute_backward")
    return dx


def _weighted(ys, rows, w, shared, gate, at):
    """Addresses of unpermute's inputs, checked: (ys, rows, w, shared, gate)."""
    import torch
    if (shared is None) != (gate is None):
        raise ValueError("shared and gate: both or neither")
    (n, H), T = ys.shape, w.shape[0]
    return (_want("ys", ys, ys.dtype, (n, H), at), _want("rows", rows, torch.int32, (T * 8,), at),
            _want("w", w, torch.float32, (T, 8), at),
            None if shared is None else _want("shared", shared, ys.dtype, (T, H), at),
            None if gate is None else _want("gate", gate, torch.float32, (T,), at))


def unpermute(ys, rows, w, shared=None, gate=None, dtype=None, y=None, stream=None):
    """y [T][H] with y[t] = sum_k w[t][k] ys[rows[8t + k]] + gate[t] shared[t]; y of `dtype`
    (by default that of ys). Differentiable in ys, w, shared and gate; the gradient of a row of ys
    that no pair names is 0."""
    import torch
    dev = ys.device
    ctx = _switched(dev, stream)
    if ctx is not None:
        with ctx:
            return unpermute(ys, rows, w, shared, gate, dtype, y)
    if (ys.requires_grad or w.requires_grad or (shared is not None and shared.requires_grad) or
            (gate is not None and gate.requires_grad)) and _recorded(y, "y"):
        from .autograd import Unpermute
        return Unpermute.apply(ys, rows, w, shared, gate, dtype)
    (n, H), T, at = ys.shape, w.shape[0], dev.index
    num = _row_enum("ys", ys.dtype)
    py, pr, pw, ps, pg = _weighted(ys, rows, w, shared, gate, at)
    if y is None:
        y = torch.empty((T, H), dtype=ys.dtype if dtype is None else dtype, device=dev)
    elif dtype is not None and y.dtype != dtype:
        raise ValueError(f"y: dtype {y.dtype}, expected {dtype}")
    _check(load().moe_unpermute(py, pr, pw, ps, pg, T, H, n, num,
                                _want("y", y, y.dtype, (T, H), at), _row_enum("y", y.dtype),
                                torch._C._cuda_getCurrentRawStream(at)), "moe_unpermute")
    return y


def unpermute_backward(dy, ys, rows, w, shared=None, gate=None, dys=None, stream=None):
    """(dys [n][H], dw [T][8], dshared [T][H] or None, dgate [T] or None): the gradients of
    unpermute. Rows of dys that no pair names keep what it held."""
    import torch
    dev = ys.device
    ctx = _switched(dev, stream)
    if ctx is not None:
        with ctx:
            return unpermute_backward(dy, ys, rows, w, shared, gate, dys)
    (n, H), T, at = ys.shape, w.shape[0], dev.index
    num, dnum = _row_enum("ys", ys.dtype), _row_enum("dy", dy.dtype)
    pd = _want("dy", dy, dy.dtype, (T, H), at)
    py, pr, pw, ps, pg = _weighted(ys, rows, w, shared, gate, at)
    if dys is None:
        dys = torch.empty((n, H), dtype=ys.dtype, device=dev)
    dw = torch.empty((T, 8), dtype=torch.float32, device=dev)
    dshared = None if shared is None else torch.empty_like(shared)
    dgate = None if shared is None else torch.empty_like(gate)
    _check(load().moe_unpermute_backward(
        pd, py, pr, pw, ps, pg, T, H, n, num, dnum, _want("dys", dys, ys.dtype, (n, H), at),
        dw.data_ptr(), None if shared is None else dshared.data_ptr(),
        None if shared is None else dgate.data_ptr(), torch._C._cuda_getCurrentRawStream(at)),
        "moe_unpermute_backward")
    return dys, dw, dshared, dgate


def quantize_i8(x, stream=None):
    """(codes [n][K] int8, scales [n] fp32) of the rows of x [n][K] (fp32 or bf16), all n of them: of a
    sorted buffer with more capacity than pairs pass the rows in use, where their number is known."""
    import torch
    dev = x.device
    ctx = _switched(dev, stream)
    if ctx is not None:
        with ctx:
            return quantize_i8(x)
    (n, K), at = x.shape, dev.index
    num = _row_enum("x", x.dtype)
    px = _want("x", x, x.dtype, (n, K), at)
    q = torch.empty((n, K), dtype=torch.int8, device=dev)
    scale = torch.empty((n,), dtype=torch.float32, device=dev)
    _check(load().moe_quantize_i8(px, n, K, num, q.data_ptr(), scale.data_ptr(),
                                  torch._C._cuda_getCurrentRawStream(at)), "moe_quantize_i8")
    return q, scale


def permute_i8(x, rows, n_rows=None, stream=None):
    """(codes [n_rows][H] int8, scales [n_rows] fp32): the rows of x [T][H] quantised and sorted,
    as permute(x, rows) followed by quantize_i8. n_rows: by default T * 8. Rows that no pair names
    are not written."""
    import torch
    dev = x.device
    ctx = _switched(dev, stream)
    if ctx is not None:
        with ctx:
            return permute_i8(x, rows, n_rows)
    (T, H), at = x.shape, dev.index
    n = T * 8 if n_rows is None else n_rows
    num = _row_enum("x", x.dtype)
    px, pr = _want("x", x, x.dtype, (T, H), at), _want("rows", rows, torch.int32, (T * 8,), at)
    q = torch.empty((n, H), dtype=torch.int8, device=dev)
    scale = torch.empty((n,), dtype=torch.float32, device=dev)
    _check(load().moe_permute_i8(px, pr, T, H, n, num, q.data_ptr(), scale.data_ptr(),
                                 torch._C._cuda_getCurrentRawStream(at)), "moe_permute_i8")
    return q, scale


def matmul_i8(x, x_scale, w, w_scale, offsets=None, swiglu=False, dtype=None, y=None, stream=None):
    """y [n][M] = x_scale[n] w_scale[e][m] sum_k x[n][k] w[e][m][k] for int8 x [n][K] and
    w [E][M][K], e the expert with offsets[e] <= n < offsets[e + 1] (offsets [E + 1] int32 on the
    device; None: w holds one matrix for all rows). swiglu: w holds gate rows, then up rows, and
    y [n][M / 2] = silu(gate) up. y of `dtype`, bf16 by default; rows of no expert keep what it
    held."""
    import torch
    dev = x.device
    ctx = _switched(dev, stream)
    if ctx is not None:
        with ctx:
            return matmul_i8(x, x_scale, w, w_scale, offsets, swiglu, dtype, y)
    (n, K), (E, M, _), at = x.shape, w.shape, dev.index
    i8, f32 = torch.int8, torch.float32
    px, ps = _want("x", x, i8, (n, K), at), _want("x_scale", x_scale, f32, (n,), at)
    pw, pc = _want("w", w, i8, (E, M, K), at), _want("w_scale", w_scale, f32, (E, M), at)
    po = None if offsets is None else _want("offsets", offsets, torch.int32, (E + 1,), at)
    Mo = M // 2 if swiglu else M
    if y is None:
        y = torch.empty((n, Mo), dtype=torch.bfloat16 if dtype is None else dtype, device=dev)
    elif dtype is not None and y.dtype != dtype:
        raise ValueError(f"y: dtype {y.dtype}, expected {dtype}")
    _check(load().moe_matmul_i8(px, ps, n, pw, pc, E, M, K, po, 1 if swiglu else 0,
                                _want("y", y, y.dtype, (n, Mo), at), _row_enum("y", y.dtype),
                                torch._C._cuda_getCurrentRawStream(at)), "moe_matmul_i8")
    return y


def device_weights(layer: dict, device="cuda") -> dict:
    """Copy a numpy layer (sparse_moe_routing_amd.inputs.make_layer) to device tensors."""
    import numpy as np
    import torch

    def dev(a):
        if a is None:
            return None
        if a.dtype == np.uint16:
            a = a.view(np.int16)
        return torch.from_numpy(np.ascontiguousarray(a)).to(device)

    return {k: dev(layer.get(k)) for k in WEIGHT_KEYS + ("x",)}


def layer_from_numpy(layer: dict, max_tokens: int, device="cuda"):
    """(MoeLayer, device tensors) for a numpy layer from sparse_moe_routing_amd.inputs."""
    w = layer["workload"]
    t = device_weights(layer, device)
    m = MoeLayer(w.hidden, w.num_experts, w.inter, w.shared_inter, max_tokens, w.dtype, t)
    return m, t
