"""Python binding of include/moe_train.h: the operators that train the block's experts,
projections and norm.

    Linear    y = act(x W^T + b) + r        forward, backward
    GatedFfn  the routed experts of a MoeSpec, or one dense gated FFN   forward, backward
    Norm      layer norm, RMS norm          forward, backward

Argument marshalling only: every step runs in the library's CUDA kernels. A handle holds the
operator's shape and one status word; weights are passed at each call (a training step changes
them), outputs and workspaces come from PyTorch's allocator at each call, so calls on several
streams and captured graphs share nothing but the status word. Tensors are [rows, width], rows
may be strided. A call runs on `stream`, or on the current stream of the handle's device; with
`stream` its tensors may be dropped at once (not with a torch.cuda.ExternalStream, whose end
PyTorch does not know), and what it returns belongs to that stream.

The calls are no autograd functions: what a forward call returns does not require a gradient,
whatever its tensors do, and the caller runs the backward calls. The router has none beyond
"topk_w".
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import Dict, Optional, Tuple

import torch

from . import inputs
from . import moe as M

# The entry points include/moe_train.h declares.
EXPORTS = [
    "moe_linear_workspace_size", "moe_linear_forward", "moe_linear_backward",
    "moe_ffn_workspace_size", "moe_ffn_dense_workspace_size", "moe_ffn_forward", "moe_ffn_backward",
    "moe_norm_workspace_size", "moe_norm_forward", "moe_norm_backward",
]

LINEAR_ACTIVATION = {"none": 0, "silu": 1, "gelu": 2}
NORM_KIND = {"layer": 0, "rms": 1}
GRAD_FIELDS = ["gate_w", "up_w", "gate_up_w", "gate_b", "up_b", "gate_up_b", "down_w", "down_b"]
_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}

# What a call needs of PyTorch's CUDA runtime, without the checks of the public wrappers (a current
# device, a stream and a workspace cost 2 us less per call). The allocator is the same one: memory
# freed after the launch is handed out again on that stream only, in a graph's pool within it.
# A PyTorch without CUDA has none of them: the module imports there too, and a handle says what is
# missing.
_current_device, _current_stream, _allocate, _free = (getattr(torch._C, n, None) for n in (
    "_cuda_getDevice", "_cuda_getCurrentRawStream", "_cuda_cudaCachingAllocator_raw_alloc",
    "_cuda_cudaCachingAllocator_raw_delete"))


class MoeLinearDesc(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class MoeNormDesc(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("kind", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class MoeFfnGrads(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in GRAD_FIELDS]


@functools.lru_cache(maxsize=None)
def lib():
    """The loaded library with this header's signatures."""
    L = M.lib()
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    szp = ctypes.POINTER(ctypes.c_size_t)
    lin, nrm = ctypes.POINTER(MoeLinearDesc), ctypes.POINTER(MoeNormDesc)
    cfg, wts, gr = ctypes.POINTER(M.MoeConfig), ctypes.POINTER(M.MoeWeights), ctypes.POINTER(MoeFfnGrads)
    sig = {
        "moe_linear_workspace_size": [lin, i64, i32, szp],
        "moe_linear_forward": [lin, vp, i64, vp, vp, vp, i64, i64, vp, i64, vp, vp, sz, vp, vp],
        "moe_linear_backward": [lin, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, sz, vp, vp],
        "moe_ffn_workspace_size": [cfg, i64, i32, szp],
        "moe_ffn_dense_workspace_size": [cfg, i64, i32, szp],
        "moe_ffn_forward": [cfg, wts, vp, i64, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, sz, vp, vp],
        "moe_ffn_backward": [cfg, wts, vp, i64, i64, vp, vp, vp, vp, vp, i64, vp, i64, vp, gr, vp, sz, vp, vp],
        "moe_norm_workspace_size": [nrm, i64, i32, szp],
        "moe_norm_forward": [nrm, vp, i64, vp, vp, i64, vp, i64, vp, vp],
        "moe_norm_backward": [nrm, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, sz, vp],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    return L


def _c_int(**sizes):
    """The C structures hold sizes in 32 bits, and ctypes drops what does not fit."""
    for name, n in sizes.items():
        if not -2 ** 31 <= n < 2 ** 31:
            raise M.MoeError(M.STATUS_CODE["MOE_ERR_SHAPE_OVERFLOW"], f"{name} = {n}")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


class _Operator:
    """What the handles share: device, dtype, status word, checks, workspace, stream.

    A call of a few microseconds on the GPU is soon bound by its Python side, so the checks
    below read each tensor attribute once and the handle keeps what does not change."""

    def __init__(self, dtype: str, device):
        if dtype not in _DTYPE:
            raise ValueError(f"dtype {dtype!r}: 'f32' or 'bf16'")
        self.dtype = _DTYPE[dtype]
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"device {device!r}: the operators run on CUDA devices")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self.lib = lib()
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._tail = (self.status.data_ptr(),)  # what follows the workspace in a call

    def device_status(self) -> int:
        """The status device-side checks left since the last call (0: none). Synchronises."""
        torch.cuda.synchronize(self.device)
        v = int(self.status.item())
        self.status.zero_()
        return v

    def _elsewhere(self, stream) -> bool:
        """Whether the call names a stream, or another device is current."""
        return stream is not None or _current_device() != self._index

    @contextlib.contextmanager
    def _on(self, stream, *tensors):
        """The handle's device and the call's stream made current: what is allocated in the
        call belongs to the stream that uses it. The caller's tensors are marked as in use on a
        stream that the call names, so that one that is dropped after the call is not handed
        out again before that stream has passed it."""
        if stream is not None:
            if stream.device != self.device:
                raise ValueError(f"stream of {stream.device}, handle of {self.device}")
            with torch.cuda.stream(stream):
                yield
            if not isinstance(stream, torch.cuda.ExternalStream):  # which may be gone when they are freed
                for t in (*tensors, self.status):
                    if t is not None:
                        t.record_stream(stream)
        else:
            with torch.cuda.device(self.device):
                yield

    def _flat(self, name: str, t: torch.Tensor, numel: int, dtype=None) -> int:
        """A contiguous tensor of a given size: its address."""
        dtype = dtype or self.dtype
        if t.dtype is not dtype or t.get_device() != self._index:
            raise ValueError(f"{name}: {t.dtype} on {t.device}, wanted {dtype} on {self.device}")
        if t.numel() != numel or not t.is_contiguous():
            raise ValueError(f"{name}: shape {tuple(t.shape)}, strides {t.stride()}; wanted {numel} contiguous values")
        return t.data_ptr()

    def _rows(self, name: str, t: torch.Tensor, width: int, rows: Optional[int] = None) -> Tuple[int, int]:
        """A [rows, width] tensor with unit column stride: its address and row stride."""
        if t.dtype is not self.dtype or t.get_device() != self._index:
            raise ValueError(f"{name}: {t.dtype} on {t.device}, wanted {self.dtype} on {self.device}")
        shape = t.shape
        if len(shape) != 2 or shape[1] != width or (rows is not None and shape[0] != rows):
            raise ValueError(f"{name}: shape {tuple(shape)}, wanted [{'rows' if rows is None else rows}, {width}]")
        n, (ld, unit) = shape[0], t.stride()
        if n and width > 1 and unit != 1:
            raise ValueError(f"{name}: strides {(ld, unit)}: the columns of a row must be contiguous")
        return t.data_ptr(), ld if n > 1 else width

    @staticmethod
    def _size(sizes, T: int, backward: int) -> int:
        """Bytes of workspace; also the library's check of the operator's shape."""
        size_fn, desc_ref, known = sizes
        out = ctypes.c_size_t(0)
        M._check(size_fn(desc_ref, T, backward, ctypes.byref(out)), size_fn.__name__)
        if len(known) >= 1024:
            known.clear()
        known[(T, backward)] = out.value
        return out.value

    def _launch(self, fn, sizes, T: int, backward: int, *args):
        """fn(desc, args, workspace, its size, status, stream) on the current stream. sizes: the call
        that says how large a workspace is, the desc, and what it said before (by tokens and direction)."""
        _, desc_ref, known = sizes
        n = known.get((T, backward))
        if n is None:
            n = self._size(sizes, T, backward)
        stream = _current_stream(self._index)
        ws = _allocate(n, stream) if n else None
        try:
            status = fn(desc_ref, *args, ws, n, *self._tail, stream)
        finally:
            if n:
                _free(ws)
        if status:
            M._check(status, fn.__name__)

    def _empty(self, *shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)

    @staticmethod
    def _like(t, shape):
        """An uninitialised tensor of t's dtype; like t where t has that shape (half a
        microsecond less than by its sizes)."""
        return torch.empty_like(t) if t.shape == shape and t.is_contiguous() else t.new_empty(shape)


class Linear(_Operator):
    """y = act(x W^T + b) + r with x [T, in], W [out, in] (moe_linear_forward / _backward)."""

    def __init__(self, in_features: int, out_features: int, activation: str = "none", dtype: str = "bf16",
                 device="cuda"):
        if activation not in LINEAR_ACTIVATION:
            raise ValueError(f"activation {activation!r}: one of {sorted(LINEAR_ACTIVATION)}")
        _c_int(in_features=in_features, out_features=out_features)
        super().__init__(dtype, device)
        self.n_in, self.n_out, self.activation = in_features, out_features, activation
        self.desc = MoeLinearDesc(in_features, out_features, LINEAR_ACTIVATION[activation], inputs.DTYPE[dtype])
        self._desc = ctypes.byref(self.desc)
        self._sizes = (self.lib.moe_linear_workspace_size, self._desc, {})
        self._size(self._sizes, 0, 0)  # checks the shape

    def forward(self, x, w, bias=None, residual=None, keep: bool = False, out=None, stream=None):
        """y, or (y, pre) with keep: pre = x W^T + b is what backward needs of an activation."""
        if self._elsewhere(stream):
            with self._on(stream, x, w, bias, residual, out):
                return self.forward(x, w, bias, residual, keep, out)
        T, K, N = x.shape[0], self.n_in, self.n_out
        xp, ldx = self._rows("x", x, K)
        wp = self._flat("w", w, N * K)
        bp = None if bias is None else self._flat("bias", bias, N)
        rp, ldr = (None, 0) if residual is None else self._rows("residual", residual, N, T)
        if out is None:
            y = self._like(x if residual is None else residual, (T, N))
            yp, ldy = y.data_ptr(), N
        else:
            y = out
            yp, ldy = self._rows("out", out, N, T)
        pre = self._empty(T, N) if keep else None
        self._launch(self.lib.moe_linear_forward, self._sizes, T, 0,
                     xp, ldx, wp, bp, rp, ldr, T, yp, ldy, _p(pre))
        return (y, pre) if keep else y

    def backward(self, dy, x, w, pre=None, bias_grad: bool = True, input_grad: bool = True,
                 weight_grad: bool = True, stream=None):
        """(dx, dw, db); None for a gradient not asked for. A residual's gradient is dy."""
        if self._elsewhere(stream):
            with self._on(stream, dy, x, w, pre):
                return self.backward(dy, x, w, pre, bias_grad, input_grad, weight_grad)
        T, K, N = x.shape[0], self.n_in, self.n_out
        gp, ldg = self._rows("dy", dy, N, T)
        xp, ldx = self._rows("x", x, K)
        wp = self._flat("w", w, N * K)
        pp = None if pre is None else self._flat("pre", pre, T * N)
        dx = self._like(x, (T, K)) if input_grad else None
        dw = self._like(w, (N, K)) if weight_grad else None
        db = self._empty(N) if bias_grad else None
        self._launch(self.lib.moe_linear_backward, self._sizes, T, 1,
                     gp, ldg, xp, ldx, wp, pp, T, _p(dx), K, _p(dw), _p(db))
        return dx, dw, db


class GatedFfn(_Operator):
    """The routed experts of a MoeSpec (f32 or bf16 planes), or, with one expert, top_k 1 and
    no routing, a dense gated FFN (moe_ffn_forward / _backward).

    weights: the planes by their moe_weights names (gate_w, up_w or gate_up_w, down_w, and the
    biases of a spec with has_expert_bias); other entries are not read. routing:
    (expert_offsets, sorted_slot, topk_w) from moe_route and moe_permute."""

    def __init__(self, spec, device="cuda"):
        _c_int(**{n: getattr(spec, n) for n in ("hidden", "latent_dim", "intermediate", "num_experts", "top_k")})
        super().__init__(spec.act_dtype, device)
        self.spec = spec
        self.cfg = M.config_from_spec(spec)
        self._cfg = ctypes.byref(self.cfg)
        M._check(M.moe_config_validate(self.cfg), "moe_config_validate")
        E, I, K = spec.num_experts, spec.intermediate, spec.expert_in
        self.E, self.k, self.I, self.K = E, spec.top_k, I, K
        self._routed = (self.lib.moe_ffn_workspace_size, self._cfg, {})
        self._dense = (self.lib.moe_ffn_dense_workspace_size, self._cfg, {})
        self._size(self._routed, 0, 0)  # checks the weight format
        shapes = {"gate_up_w": (E, 2 * I, K)} if spec.gate_up_interleaved else {"gate_w": (E, I, K), "up_w": (E, I, K)}
        shapes["down_w"] = (E, K, I)
        if spec.has_expert_bias:
            shapes.update({"gate_up_b": (E, 2 * I)} if spec.gate_up_interleaved else {"gate_b": (E, I), "up_b": (E, I)})
            shapes["down_b"] = (E, K)
        self.shapes = shapes
        self._planes_numel = [(f, functools.reduce(int.__mul__, s)) for f, s in shapes.items()]

    def _used(self, tensors):
        """The entries of a dict of planes that the calls read."""
        return [tensors.get(f) for f in self.shapes]

    def _planes(self, tensors):
        w, dtype, index = M.MoeWeights(), self.dtype, self._index
        for f, n in self._planes_numel:
            t = tensors.get(f)
            if t is None:
                raise M.MoeError(M.STATUS_CODE["MOE_ERR_MISSING_TENSOR"], f"weights {f}")
            if t.dtype is not dtype or t.get_device() != index or t.numel() != n or not t.is_contiguous():
                self._flat(f, t, n)  # says what is wrong
            setattr(w, f, t.data_ptr())
        return w

    def _routing(self, routing, T: int):
        if routing is None:
            if self.E != 1 or self.k != 1:
                raise ValueError(f"{self.E} experts, top_k {self.k}: routing is needed")
            return None, None, None
        off, slots, wts = routing
        return (self._flat("expert_offsets", off, self.E + 1, torch.int32),
                self._flat("sorted_slot", slots, T * self.k, torch.int32),
                self._flat("topk_w", wts, T * self.k, torch.float32))

    def forward(self, u, weights: Dict[str, torch.Tensor], routing=None, residual=None, keep: bool = True,
                out=None, stream=None):
        """(y, pre): y [T, K], and the pre-activations [T*k, 2I] in sorted order that backward
        takes (None without keep)."""
        if self._elsewhere(stream):
            with self._on(stream, u, *self._used(weights), *(routing or ()), residual, out):
                return self.forward(u, weights, routing, residual, keep, out)
        T = u.shape[0]
        up, ldu = self._rows("u", u, self.K)
        w = self._planes(weights)
        off, slots, wts = self._routing(routing, T)
        rp, ldr = (None, 0) if residual is None else self._rows("residual", residual, self.K, T)
        if out is None:
            y = self._like(u, (T, self.K))
            yp, ldy = y.data_ptr(), self.K
        else:
            y = out
            yp, ldy = self._rows("out", out, self.K, T)
        pre = self._empty(T * self.k, 2 * self.I) if keep else None
        self._launch(self.lib.moe_ffn_forward, self._dense if routing is None else self._routed, T, 0,
                     ctypes.byref(w), up, ldu, T, off, slots, wts, rp, ldr, yp, ldy, _p(pre))
        return y, pre

    def backward(self, dy, u, weights: Dict[str, torch.Tensor], pre, routing=None, input_grad: bool = True,
                 stream=None) -> Dict[str, torch.Tensor]:
        """Gradients by name: "x" (of u), "topk_w" (routed), and those of the weight planes."""
        if self._elsewhere(stream):
            with self._on(stream, dy, u, *self._used(weights), pre, *(routing or ())):
                return self.backward(dy, u, weights, pre, routing, input_grad)
        T = u.shape[0]
        gp, ldg = self._rows("dy", dy, self.K, T)
        up, ldu = self._rows("u", u, self.K)
        w = self._planes(weights)
        off, slots, wts = self._routing(routing, T)
        pp = self._flat("pre", pre, T * self.k * 2 * self.I)
        grads = {f: self._like(weights[f], s) for f, s in self.shapes.items()}
        g = MoeFfnGrads()
        for f, t in grads.items():
            setattr(g, f, t.data_ptr())
        dwt = None if off is None else self._empty(T, self.k, dtype=torch.float32)
        du = self._like(u, (T, self.K)) if input_grad else None
        self._launch(self.lib.moe_ffn_backward, self._dense if routing is None else self._routed, T, 1,
                     ctypes.byref(w), up, ldu, T, off, slots, wts, pp, gp, ldg, _p(du), self.K, _p(dwt),
                     ctypes.byref(g))
        if du is not None:
            grads["x"] = du
        if dwt is not None:
            grads["topk_w"] = dwt
        return grads


class Norm(_Operator):
    """Layer norm or RMS norm over the last axis (moe_norm_forward / _backward)."""

    def __init__(self, width: int, kind: str = "rms", eps: float = 1e-6, dtype: str = "bf16", device="cuda"):
        if kind not in NORM_KIND:
            raise ValueError(f"kind {kind!r}: one of {sorted(NORM_KIND)}")
        _c_int(width=width)
        super().__init__(dtype, device)
        self.width, self.kind = width, kind
        self.desc = MoeNormDesc(width, NORM_KIND[kind], inputs.DTYPE[dtype], eps)
        self._desc = ctypes.byref(self.desc)
        self._sizes = (self.lib.moe_norm_workspace_size, self._desc, {})
        self._size(self._sizes, 0, 0)  # checks the shape
        self._tail = ()  # these calls take no status

    def forward(self, x, w, bias=None, out=None, stream=None):
        """(y, stats): stats [T, 2] f32 (mean, 1 / sqrt(var + eps)) is what backward takes."""
        if self._elsewhere(stream):
            with self._on(stream, x, w, bias, out):
                return self.forward(x, w, bias, out)
        T, H = x.shape[0], self.width
        xp, ldx = self._rows("x", x, H)
        wp = self._flat("w", w, H)
        bp = None if bias is None else self._flat("bias", bias, H)
        if out is None:
            y = self._like(x, (T, H))
            yp, ldy = y.data_ptr(), H
        else:
            y = out
            yp, ldy = self._rows("out", out, H, T)
        stats = self._empty(T, 2, dtype=torch.float32)
        M._check(self.lib.moe_norm_forward(self._desc, xp, ldx, wp, bp, T, yp, ldy, stats.data_ptr(),
                                           _current_stream(self._index)), "moe_norm_forward")
        return y, stats

    def backward(self, dy, x, w, stats, bias_grad: Optional[bool] = None, input_grad: bool = True,
                 stream=None):
        """(dx, dw, db); db is None for RMS norm or with bias_grad False."""
        if self._elsewhere(stream):
            with self._on(stream, dy, x, w, stats):
                return self.backward(dy, x, w, stats, bias_grad, input_grad)
        T, H = x.shape[0], self.width
        if bias_grad and self.kind == "rms":
            raise ValueError("RMS norm has no bias")
        if bias_grad is None:
            bias_grad = self.kind == "layer"
        gp, ldg = self._rows("dy", dy, H, T)
        xp, ldx = self._rows("x", x, H)
        wp = self._flat("w", w, H)
        sp = self._flat("stats", stats, 2 * T, torch.float32)
        dx = self._like(x, (T, H)) if input_grad else None
        dw = self._like(w, (H,))
        db = self._like(w, (H,)) if bias_grad else None
        self._launch(self.lib.moe_norm_backward, self._sizes, T, 1,
                     gp, ldg, xp, ldx, wp, sp, T, _p(dx), H, _p(dw), _p(db))
        return dx, dw, db
