"""Fused LoRA / QLoRA projections for AMD MI355X (gfx950).

Thin Python layer over the C-ABI library ``liblora_mi355x.so``: it allocates
outputs and workspace with PyTorch (device memory and streams only), fills
the C descriptors and calls the library.  All arithmetic runs in the
library's HIP kernels.

Layouts follow the C header: W [n_in, n_out], A [n_in, r], B [r, n_out],
row-major; bf16 or fp32 compute; NF4 bases in bf16.  bf16 inputs with fp32
adapters select the fp32 LoRA-gradient mode (fp32 dA, dB).

Beside the projections: ``multi_fwd`` (rows of one batch with different
adapters), ``block_norm_fwd`` / ``block_norm_bwd`` (norms before and after a
block with its gate and residual) and ``orthogonalize`` / ``muon_step``
(orthogonalised updates of the adapters).  These run on the device of their
tensors, current or not, on ``stream`` or that device's current stream, and
can be captured into a graph; a workspace given as ``ws`` must not be in use
by another call at the same time.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import functools
from dataclasses import dataclass
from typing import Optional

from . import _lib as L

__all__ = [
    "Proj", "NF4Weight", "load", "LoraError",
    "mlp_fwd", "mlp_bwd", "mlp_workspace_size",
    "relu2_mlp_fwd", "relu2_mlp_bwd", "relu2_mlp_workspace_size",
    "qkv_fwd", "qkv_bwd", "o_fwd", "o_bwd", "o_fwd_noalloc",
    "AdapterPool", "multi_fwd", "multi_workspace_size",
    "block_norm_fwd", "block_norm_bwd", "block_norm_workspace_size",
    "orthogonalize", "muon_step", "orth_workspace_size",
    "nf4_quantize", "nf4_dequant", "nf4_unpack_codes", "nf4_gemm", "nf4_codebook",
    "trace_begin", "trace_end",
]

load = L.load
LoraError = L.LoraError


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return L.LORA_BF16
    if t.dtype == torch.float32:
        return L.LORA_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _call_dtype(X, projs) -> int:
    """dtype code of a call: X's dtype, or the fp32 LoRA-gradient mode
    (LORA_BF16_F32LORA) when X is bf16 and the adapters are fp32.  Dense
    bases must have X's dtype."""
    torch = _torch()
    ad = {t.dtype for p in projs for t in (p.A, p.B)}
    if len(ad) != 1:
        raise ValueError(f"the adapters of one call must share a dtype, got {sorted(map(str, ad))}")
    for p in projs:
        if p.W is not None and p.W.dtype != X.dtype:
            raise ValueError(f"base weight dtype {p.W.dtype} differs from the input dtype {X.dtype}")
    (a,) = ad
    if a == X.dtype:
        return _dtype_code(X)
    if X.dtype == torch.bfloat16 and a == torch.float32:
        return L.LORA_BF16_F32LORA
    raise ValueError(f"adapters in {a} with inputs in {X.dtype} are not supported")


def _stream(stream) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ws(nbytes: int, device):
    torch = _torch()
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _nbytes(ws, device) -> int:
    """Size in bytes of a caller's workspace tensor (dense, on the call's device)."""
    if not ws.is_contiguous():
        raise ValueError("ws is not contiguous")
    if ws.device != device:
        raise ValueError(f"ws is on {ws.device}, expected {device}")
    return ws.numel() * ws.element_size()


def _set_plan(desc, plan):
    """Put an optional GEMM launch plan into a call descriptor: a sequence of
    up to two (group, ksplit) pairs, the call's GEMMs in launch order (see
    lora_plan in the C header); None keeps the library's defaults.  The
    ctypes pointer keeps the struct alive as long as the descriptor."""
    if plan is None:
        return desc
    entries = list(plan)
    if len(entries) > 2:
        raise ValueError(f"a plan has at most two GEMM entries, got {len(entries)}")
    p = L.lora_plan()
    for i, e in enumerate(entries):
        g, k = (int(x) for x in e)
        p.gemm[i].group, p.gemm[i].ksplit = g, k
    desc.plan = C.pointer(p)
    return desc


_NO_STREAM = contextlib.nullcontext()


def _on(stream):
    """Allocation context of a call: PyTorch's caching allocator ties every
    tensor allocated inside it (outputs, workspace) to the stream the library
    enqueues on, so a buffer is not handed to other work while the call's
    kernels may still use it."""
    return _NO_STREAM if stream is None else _torch().cuda.stream(stream)


def _need(name, t, shape, dtype, device):
    """Raise ValueError unless t is a dense tensor of this shape and dtype on
    this device (the kernels take row-major dense buffers)."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.shape != shape and tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(int(x) for x in shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous (the library takes dense row-major buffers)")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device} (the device of X)")


def _on_gpu(X, ws=None):
    if ws is not None:
        _nbytes(ws, X.device)
    if X.device.type != "cuda":
        raise ValueError(f"X is on {X.device}: the library runs on the GPU only")


def _x2d(name, X):
    if X.dim() != 2:
        raise ValueError(f"{name} must be 2-D [tokens, width], got shape {tuple(X.shape)}")
    return X.shape


def _adapter_dtype(X, dt):
    torch = _torch()
    return torch.float32 if dt in (L.LORA_F32, L.LORA_BF16_F32LORA) else X.dtype


def _check_proj(name, p, n_in, n_out, r, X, dt):
    """A [n_in, r], B [r, n_out] in the call's adapter dtype; the base W
    [n_in, n_out] in X's dtype, or an NF4 weight of that shape."""
    torch = _torch()
    ad = _adapter_dtype(X, dt)
    _need(f"{name}.A", p.A, (n_in, r), ad, X.device)
    _need(f"{name}.B", p.B, (r, n_out), ad, X.device)
    if (p.W is None) == (p.nf4 is None):
        raise ValueError(f"{name}: exactly one of W and nf4 must be set")
    if p.Wt is not None:
        if p.W is None:
            raise ValueError(f"{name}: Wt is only for a dense W")
        _need(f"{name}.Wt", p.Wt, (n_out, n_in), X.dtype, X.device)
    if p.W is not None:
        _need(f"{name}.W", p.W, (n_in, n_out), X.dtype, X.device)
    else:
        w = p.nf4
        if (w.rows, w.cols) != (n_in, n_out):
            raise ValueError(f"{name}: NF4 weight is [{w.rows}, {w.cols}], expected [{n_in}, {n_out}]")
        _check_nf4(name, w, X.device)


def _check_nf4(name, w, device):
    torch = _torch()
    n = w.rows * w.cols
    if n % (64 * 256):
        raise ValueError(f"{name}: NF4 element count {n} is not a multiple of {64 * 256}")
    _need(f"{name}.codes", w.codes, (n // 2,), torch.uint8, device)
    _need(f"{name}.q8", w.q8, (n // 64,), torch.int8, device)
    _need(f"{name}.s2", w.s2, (n // (64 * 256),), torch.float32, device)
    _need(f"{name}.mu", w.mu, (1,), torch.float32, device)


@dataclass
class NF4Weight:
    """NF4-packed weight W [rows, cols] (device tensors)."""

    codes: object  # uint8 [numel/2]
    q8: object     # int8 [numel/64]
    s2: object     # float32 [numel/16384]
    mu: object     # float32 [1]
    rows: int
    cols: int

    def c_struct(self) -> L.lora_nf4:
        return L.lora_nf4(_ptr(self.codes), _ptr(self.q8), _ptr(self.s2), _ptr(self.mu), self.rows, self.cols)


@dataclass
class Proj:
    """One LoRA projection: dense W or NF4 weight, adapters A, B and scale s.
    Wt (optional, dense bf16 only): the same weight stored [n_out, n_in]
    (W.t().contiguous(), PyTorch nn.Linear's layout); the forward GEMMs read
    it when every projection they read has one."""

    A: object
    B: object
    scale: float
    W: object = None
    nf4: Optional[NF4Weight] = None
    Wt: object = None

    def c_struct(self, keep: list) -> L.lora_proj:
        p = L.lora_proj()
        p.W = _ptr(self.W)
        if self.nf4 is not None:
            s = self.nf4.c_struct()
            keep.append(s)
            p.nf4 = C.pointer(s)
        p.A = _ptr(self.A)
        p.B = _ptr(self.B)
        p.scale = float(self.scale)
        p.Wt = _ptr(self.Wt)
        return p


# ---------------------------------------------------------------------------
# MLP
# ---------------------------------------------------------------------------

def mlp_workspace_size(T, H, I, r, act="swiglu", dtype=L.LORA_BF16, plan=None):
    d = _set_plan(L.lora_mlp_desc(T, H, I, r, L.ACT_CODES[act], dtype), plan)
    f, b = C.c_size_t(), C.c_size_t()
    L.call("lora_mlp_workspace_size", C.byref(d), C.byref(f), C.byref(b))
    return f.value, b.value


def _mlp_dims(X, gate, up, down):
    T, H = _x2d("X", X)
    if gate.A.dim() != 2 or gate.B.dim() != 2:
        raise ValueError("gate.A and gate.B must be 2-D")
    I, r = gate.B.shape[1], gate.A.shape[1]
    dt = _call_dtype(X, (gate, up, down))
    for name, p, n_in, n_out in (("gate", gate, H, I), ("up", up, H, I), ("down", down, I, H)):
        _check_proj(name, p, n_in, n_out, r, X, dt)
    return T, H, I, r, dt


def _check_saved(saved, names_shapes, X):
    if not isinstance(saved, dict):
        raise ValueError("saved must be the dict the forward returned")
    for k, shape in names_shapes:
        _need(f"saved[{k!r}]", saved.get(k), shape, X.dtype, X.device)


def mlp_fwd(X, gate: Proj, up: Proj, down: Proj, act="swiglu", *, Y=None, saved=None, ws=None, stream=None,
            plan=None):
    """Y = down(phi(gate(X)) * up(X)).  Returns (Y, saved) with saved = dict(e, g, U).

    Outputs and workspace the caller does not pass are allocated on ``stream``
    (default: the current stream), where the library enqueues its kernels."""
    torch = _torch()
    T, H, I, r, dt = _mlp_dims(X, gate, up, down)
    if act not in L.ACT_CODES:
        raise ValueError(f"unknown activation {act!r}")
    if Y is not None:
        _need("Y", Y, (T, H), X.dtype, X.device)
    if saved is not None:
        _check_saved(saved, (("e", (T, I)), ("g", (T, I)), ("U", (T, 3 * r))), X)
    _on_gpu(X, ws)
    d = _set_plan(L.lora_mlp_desc(T, H, I, r, L.ACT_CODES[act], dt), plan)
    fb, _ = mlp_workspace_size(T, H, I, r, act, dt, plan)
    with _on(stream):
        if Y is None:
            Y = torch.empty((T, H), dtype=X.dtype, device=X.device)
        if saved is None:
            saved = dict(e=torch.empty((T, I), dtype=X.dtype, device=X.device),
                         g=torch.empty((T, I), dtype=X.dtype, device=X.device),
                         U=torch.empty((T, 3 * r), dtype=X.dtype, device=X.device))
        if ws is None:
            ws = _ws(fb, X.device)
    keep = []
    sv = L.lora_mlp_saved(_ptr(saved["e"]), _ptr(saved["g"]), _ptr(saved["U"]))
    L.call("lora_mlp_fwd", C.byref(d), _ptr(X), C.byref(gate.c_struct(keep)), C.byref(up.c_struct(keep)),
           C.byref(down.c_struct(keep)), _ptr(Y), C.byref(sv), _ptr(ws), _nbytes(ws, X.device), _stream(stream))
    return Y, saved


_MLP_GRAD_KEYS = ("dA_gate", "dB_gate", "dA_up", "dB_up", "dA_down", "dB_down")


def mlp_bwd(dY, X, saved, gate: Proj, up: Proj, down: Proj, act="swiglu", *, dX=None, grads=None, ws=None,
            stream=None, plan=None):
    """Returns (dX, grads) with grads = dict(dA_gate, dB_gate, dA_up, dB_up, dA_down, dB_down).
    ``dX=X`` writes the input gradient over X."""
    torch = _torch()
    T, H, I, r, dt = _mlp_dims(X, gate, up, down)
    if act not in L.ACT_CODES:
        raise ValueError(f"unknown activation {act!r}")
    _need("dY", dY, (T, H), X.dtype, X.device)
    _check_saved(saved, (("e", (T, I)), ("g", (T, I)), ("U", (T, 3 * r))), X)
    if dX is not None:
        _need("dX", dX, (T, H), X.dtype, X.device)
    if grads is not None:
        for k, p, ab in zip(_MLP_GRAD_KEYS, (gate, gate, up, up, down, down), "ABABAB"):
            ref = getattr(p, ab)
            _need(f"grads[{k!r}]", grads.get(k), ref.shape, ref.dtype, X.device)
    _on_gpu(X, ws)
    d = _set_plan(L.lora_mlp_desc(T, H, I, r, L.ACT_CODES[act], dt), plan)
    _, bb = mlp_workspace_size(T, H, I, r, act, dt, plan)
    with _on(stream):
        if dX is None:
            dX = torch.empty_like(X)
        if grads is None:
            grads = dict(dA_gate=torch.empty_like(gate.A), dB_gate=torch.empty_like(gate.B),
                         dA_up=torch.empty_like(up.A), dB_up=torch.empty_like(up.B),
                         dA_down=torch.empty_like(down.A), dB_down=torch.empty_like(down.B))
        if ws is None:
            ws = _ws(bb, X.device)
    keep = []
    sv = L.lora_mlp_saved(_ptr(saved["e"]), _ptr(saved["g"]), _ptr(saved["U"]))
    gr = L.lora_mlp_grads(*(_ptr(grads[k]) for k in _MLP_GRAD_KEYS))
    L.call("lora_mlp_bwd", C.byref(d), _ptr(dY), _ptr(X), C.byref(sv), C.byref(gate.c_struct(keep)),
           C.byref(up.c_struct(keep)), C.byref(down.c_struct(keep)), _ptr(dX), C.byref(gr), _ptr(ws),
           _nbytes(ws, X.device), _stream(stream))
    return dX, grads


# ---------------------------------------------------------------------------
# Ungated ReLU^2 MLP
# ---------------------------------------------------------------------------

def relu2_mlp_workspace_size(T, H, I, r, dtype=L.LORA_BF16, plan=None):
    d = _set_plan(L.lora_relu2_mlp_desc(T, H, I, r, dtype, 0), plan)
    f, b = C.c_size_t(), C.c_size_t()
    L.call("lora_relu2_mlp_workspace_size", C.byref(d), C.byref(f), C.byref(b))
    return f.value, b.value


def _relu2_dims(X, up, down):
    T, H = _x2d("X", X)
    if up.A.dim() != 2 or up.B.dim() != 2:
        raise ValueError("up.A and up.B must be 2-D")
    I, r = up.B.shape[1], up.A.shape[1]
    dt = _call_dtype(X, (up, down))
    _check_proj("up", up, H, I, r, X, dt)
    _check_proj("down", down, I, H, r, X, dt)
    return T, H, I, r, dt


def relu2_mlp_fwd(X, up: Proj, down: Proj, *, Y=None, saved=None, ws=None, stream=None, plan=None):
    """Y = down(relu(up(X))^2).  Returns (Y, saved) with saved = dict(u, U)."""
    torch = _torch()
    T, H, I, r, dt = _relu2_dims(X, up, down)
    if Y is not None:
        _need("Y", Y, (T, H), X.dtype, X.device)
    if saved is not None:
        _check_saved(saved, (("u", (T, I)), ("U", (T, 2 * r))), X)
    _on_gpu(X, ws)
    d = _set_plan(L.lora_relu2_mlp_desc(T, H, I, r, dt, 0), plan)
    fb, _ = relu2_mlp_workspace_size(T, H, I, r, dt, plan)
    with _on(stream):
        if Y is None:
            Y = torch.empty((T, H), dtype=X.dtype, device=X.device)
        if saved is None:
            saved = dict(u=torch.empty((T, I), dtype=X.dtype, device=X.device),
                         U=torch.empty((T, 2 * r), dtype=X.dtype, device=X.device))
        if ws is None:
            ws = _ws(fb, X.device)
    keep = []
    sv = L.lora_relu2_mlp_saved(_ptr(saved["u"]), _ptr(saved["U"]))
    L.call("lora_relu2_mlp_fwd", C.byref(d), _ptr(X), C.byref(up.c_struct(keep)), C.byref(down.c_struct(keep)),
           _ptr(Y), C.byref(sv), _ptr(ws), _nbytes(ws, X.device), _stream(stream))
    return Y, saved


_RELU2_GRAD_KEYS = ("dA_up", "dB_up", "dA_down", "dB_down")


def relu2_mlp_bwd(dY, X, saved, up: Proj, down: Proj, *, dX=None, grads=None, ws=None, stream=None, plan=None):
    """Returns (dX, grads) with grads = dict(dA_up, dB_up, dA_down, dB_down)."""
    torch = _torch()
    T, H, I, r, dt = _relu2_dims(X, up, down)
    _need("dY", dY, (T, H), X.dtype, X.device)
    _check_saved(saved, (("u", (T, I)), ("U", (T, 2 * r))), X)
    if dX is not None:
        _need("dX", dX, (T, H), X.dtype, X.device)
    if grads is not None:
        for k, p, ab in zip(_RELU2_GRAD_KEYS, (up, up, down, down), "ABAB"):
            ref = getattr(p, ab)
            _need(f"grads[{k!r}]", grads.get(k), ref.shape, ref.dtype, X.device)
    _on_gpu(X, ws)
    d = _set_plan(L.lora_relu2_mlp_desc(T, H, I, r, dt, 0), plan)
    _, bb = relu2_mlp_workspace_size(T, H, I, r, dt, plan)
    with _on(stream):
        if dX is None:
            dX = torch.empty_like(X)
        if grads is None:
            grads = dict(dA_up=torch.empty_like(up.A), dB_up=torch.empty_like(up.B),
                         dA_down=torch.empty_like(down.A), dB_down=torch.empty_like(down.B))
        if ws is None:
            ws = _ws(bb, X.device)
    keep = []
    sv = L.lora_relu2_mlp_saved(_ptr(saved["u"]), _ptr(saved["U"]))
    gr = L.lora_relu2_mlp_grads(*(_ptr(grads[k]) for k in _RELU2_GRAD_KEYS))
    L.call("lora_relu2_mlp_bwd", C.byref(d), _ptr(dY), _ptr(X), C.byref(sv), C.byref(up.c_struct(keep)),
           C.byref(down.c_struct(keep)), _ptr(dX), C.byref(gr), _ptr(ws), _nbytes(ws, X.device), _stream(stream))
    return dX, grads


# ---------------------------------------------------------------------------
# Q/K/V and O
# ---------------------------------------------------------------------------

def qkv_workspace_size(T, H, Nq, Nk, Nv, r, dtype=L.LORA_BF16, plan=None):
    d = _set_plan(L.lora_qkv_desc(T, H, Nq, Nk, Nv, r, dtype, 0), plan)
    f, b = C.c_size_t(), C.c_size_t()
    L.call("lora_qkv_workspace_size", C.byref(d), C.byref(f), C.byref(b))
    return f.value, b.value


def _qkv_dims(X, q, k, v):
    T, H = _x2d("X", X)
    if q.A.dim() != 2 or any(p.B.dim() != 2 for p in (q, k, v)):
        raise ValueError("adapters must be 2-D")
    Ns = [p.B.shape[1] for p in (q, k, v)]
    r = q.A.shape[1]
    dt = _call_dtype(X, (q, k, v))
    for name, p, n in zip("qkv", (q, k, v), Ns):
        _check_proj(name, p, H, n, r, X, dt)
    return T, H, Ns, r, dt


_QKV_GRAD_KEYS = ("dA_q", "dB_q", "dA_k", "dB_k", "dA_v", "dB_v")


def qkv_fwd(X, q: Proj, k: Proj, v: Proj, *, out=None, U=None, ws=None, stream=None, plan=None):
    """Returns (Q, K, V, U) with U = [X A_q | X A_k | X A_v]."""
    torch = _torch()
    T, H, Ns, r, dt = _qkv_dims(X, q, k, v)
    if out is not None:
        if len(out) != 3:
            raise ValueError("out must hold three tensors (Q, K, V)")
        for name, t, n in zip("QKV", out, Ns):
            _need(name, t, (T, n), X.dtype, X.device)
    if U is not None:
        _need("U", U, (T, 3 * r), X.dtype, X.device)
    _on_gpu(X, ws)
    d = _set_plan(L.lora_qkv_desc(T, H, Ns[0], Ns[1], Ns[2], r, dt, 0), plan)
    fb, _ = qkv_workspace_size(T, H, *Ns, r, dt, plan)
    with _on(stream):
        if out is None:
            out = [torch.empty((T, n), dtype=X.dtype, device=X.device) for n in Ns]
        if U is None:
            U = torch.empty((T, 3 * r), dtype=X.dtype, device=X.device)
        if ws is None:
            ws = _ws(fb, X.device)
    keep = []
    L.call("lora_qkv_fwd", C.byref(d), _ptr(X), C.byref(q.c_struct(keep)), C.byref(k.c_struct(keep)),
           C.byref(v.c_struct(keep)), _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _ptr(U), _ptr(ws), _nbytes(ws, X.device),
           _stream(stream))
    return out[0], out[1], out[2], U


def qkv_bwd(dQ, dK, dV, X, U, q: Proj, k: Proj, v: Proj, *, dX=None, grads=None, ws=None, stream=None,
            plan=None):
    """Returns (dX, grads) with grads = dict(dA_q, dB_q, dA_k, dB_k, dA_v, dB_v).
    ``dX=X`` writes the input gradient over X."""
    torch = _torch()
    T, H, Ns, r, dt = _qkv_dims(X, q, k, v)
    for name, t, n in (("dQ", dQ, Ns[0]), ("dK", dK, Ns[1]), ("dV", dV, Ns[2])):
        _need(name, t, (T, n), X.dtype, X.device)
    _need("U", U, (T, 3 * r), X.dtype, X.device)
    if dX is not None:
        _need("dX", dX, (T, H), X.dtype, X.device)
    if grads is not None:
        for key, p, ab in zip(_QKV_GRAD_KEYS, (q, q, k, k, v, v), "ABABAB"):
            ref = getattr(p, ab)
            _need(f"grads[{key!r}]", grads.get(key), ref.shape, ref.dtype, X.device)
    _on_gpu(X, ws)
    d = _set_plan(L.lora_qkv_desc(T, H, Ns[0], Ns[1], Ns[2], r, dt, 0), plan)
    _, bb = qkv_workspace_size(T, H, *Ns, r, dt, plan)
    with _on(stream):
        if dX is None:
            dX = torch.empty_like(X)
        if grads is None:
            grads = dict(dA_q=torch.empty_like(q.A), dB_q=torch.empty_like(q.B), dA_k=torch.empty_like(k.A),
                         dB_k=torch.empty_like(k.B), dA_v=torch.empty_like(v.A), dB_v=torch.empty_like(v.B))
        if ws is None:
            ws = _ws(bb, X.device)
    keep = []
    gr = L.lora_qkv_grads(*(_ptr(grads[n]) for n in _QKV_GRAD_KEYS))
    L.call("lora_qkv_bwd", C.byref(d), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(X), _ptr(U), C.byref(q.c_struct(keep)),
           C.byref(k.c_struct(keep)), C.byref(v.c_struct(keep)), _ptr(dX), C.byref(gr), _ptr(ws), _nbytes(ws, X.device),
           _stream(stream))
    return dX, grads


def o_workspace_size(T, K, N, r, dtype=L.LORA_BF16, plan=None):
    d = _set_plan(L.lora_o_desc(T, K, N, r, dtype, 0), plan)
    f, b = C.c_size_t(), C.c_size_t()
    L.call("lora_o_workspace_size", C.byref(d), C.byref(f), C.byref(b))
    return f.value, b.value


def _o_dims(X, o):
    T, K = _x2d("X", X)
    if o.A.dim() != 2 or o.B.dim() != 2:
        raise ValueError("o.A and o.B must be 2-D")
    N, r = o.B.shape[1], o.A.shape[1]
    dt = _call_dtype(X, (o,))
    _check_proj("o", o, K, N, r, X, dt)
    return T, K, N, r, dt


def o_fwd(X, o: Proj, *, Y=None, U=None, ws=None, stream=None, plan=None):
    """Returns (Y, U)."""
    torch = _torch()
    T, K, N, r, dt = _o_dims(X, o)
    if Y is not None:
        _need("Y", Y, (T, N), X.dtype, X.device)
    if U is not None:
        _need("U", U, (T, r), X.dtype, X.device)
    _on_gpu(X, ws)
    d = _set_plan(L.lora_o_desc(T, K, N, r, dt, 0), plan)
    fb, _ = o_workspace_size(T, K, N, r, dt, plan)
    with _on(stream):
        if Y is None:
            Y = torch.empty((T, N), dtype=X.dtype, device=X.device)
        if U is None:
            U = torch.empty((T, r), dtype=X.dtype, device=X.device)
        if ws is None:
            ws = _ws(fb, X.device)
    keep = []
    L.call("lora_o_fwd", C.byref(d), _ptr(X), C.byref(o.c_struct(keep)), _ptr(Y), _ptr(U), _ptr(ws), _nbytes(ws, X.device),
           _stream(stream))
    return Y, U


def o_fwd_noalloc(X, o: Proj, *, Y, U, stream=None, plan=None):
    """o_fwd for callers that cannot allocate: the library takes its scratch
    from a static per-GPU array (at most NOALLOC_SCRATCH_BYTES, shared by all
    such calls on that GPU) and allocates nothing; the caller passes the
    outputs Y [T, N] and U [T, r].  Returns (Y, U)."""
    T, K, N, r, dt = _o_dims(X, o)
    _need("Y", Y, (T, N), X.dtype, X.device)
    _need("U", U, (T, r), X.dtype, X.device)
    _on_gpu(X)
    d = _set_plan(L.lora_o_desc(T, K, N, r, dt, 0), plan)
    keep = []
    L.call("lora_o_fwd_noalloc", C.byref(d), _ptr(X), C.byref(o.c_struct(keep)), _ptr(Y), _ptr(U),
           _stream(stream))
    return Y, U


NOALLOC_SCRATCH_BYTES = L.NOALLOC_SCRATCH_BYTES


def o_bwd(dY, X, U, o: Proj, *, dX=None, dA=None, dB=None, ws=None, stream=None, plan=None):
    """Returns (dX, dA, dB).  ``dX=X`` writes the input gradient over X."""
    torch = _torch()
    T, K, N, r, dt = _o_dims(X, o)
    _need("dY", dY, (T, N), X.dtype, X.device)
    _need("U", U, (T, r), X.dtype, X.device)
    if dX is not None:
        _need("dX", dX, (T, K), X.dtype, X.device)
    if dA is not None:
        _need("dA", dA, o.A.shape, o.A.dtype, X.device)
    if dB is not None:
        _need("dB", dB, o.B.shape, o.B.dtype, X.device)
    _on_gpu(X, ws)
    d = _set_plan(L.lora_o_desc(T, K, N, r, dt, 0), plan)
    _, bb = o_workspace_size(T, K, N, r, dt, plan)
    with _on(stream):
        dX = torch.empty_like(X) if dX is None else dX
        dA = torch.empty_like(o.A) if dA is None else dA
        dB = torch.empty_like(o.B) if dB is None else dB
        if ws is None:
            ws = _ws(bb, X.device)
    keep = []
    L.call("lora_o_bwd", C.byref(d), _ptr(dY), _ptr(X), _ptr(U), C.byref(o.c_struct(keep)), _ptr(dX), _ptr(dA),
           _ptr(dB), _ptr(ws), _nbytes(ws, X.device), _stream(stream))
    return dX, dA, dB


# ---------------------------------------------------------------------------
# Adapters of many requests beside one shared projection
# ---------------------------------------------------------------------------

def _current_stream(dev) -> int:
    """The current stream of a device as the library takes it.  torch's internal accessor takes 0.1 us, the
    public stream object 1.9 (a tenth of a small call); where a torch build lacks the first, the second serves."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev.index) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _call_on(t, stream, name, *args):
    """L.call(name, *args, stream) on t's device, with the given stream or that
    device's current one."""
    torch = _torch()
    dev = t.device
    if stream is None:
        raw = _current_stream(dev)
    elif stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, expected {dev}")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == dev.index:
        L.call(name, *args, raw)
    else:
        with torch.cuda.device(dev):
            L.call(name, *args, raw)


def _ws_for(ws, need, dev):
    """The workspace of a call and its size: the caller's (as _on_gpu has checked it) or a new one."""
    if ws is not None:
        return ws, ws.numel() * ws.element_size()
    return _torch().empty(need or 1, dtype=_torch().uint8, device=dev), need


@dataclass
class AdapterPool:
    """Adapters of one projection, stacked: A [n, n_in, r], B [n, r, n_out] and their scales [n] (fp32).
    A and B have the type of the activations (adapters trained in fp32 beside bf16 are cast once, here)."""

    A: object
    B: object
    scale: object


@functools.lru_cache(maxsize=1024)
def multi_workspace_size(T, K, N, r, n, dtype=L.LORA_BF16):
    d = L.lora_multi_desc(T, K, N, r, n, dtype, 0)
    b = C.c_size_t()
    L.call("lora_multi_workspace_size", C.byref(d), C.byref(b))
    return b.value


def multi_fwd(X, W, pool: AdapterPool, ids, *, Y=None, ws=None, stream=None):
    """Y[t] = X[t] W + scale[i] (X[t] A[i]) B[i] with i = ids[t], for X [T, n_in], W [n_in, n_out] and ids [T]
    (int32, on the GPU, rows in any order); a row whose id is outside [0, n) takes the base alone.

    With W None the adapter terms are added to Y in place: Y then holds the product with a base kept in another
    form (``nf4_gemm``).  Returns Y."""
    torch = _torch()
    T, K = _x2d("X", X)
    A, B, dtype, dev = pool.A, pool.B, X.dtype, X.device
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("pool.A must be [n, n_in, r] and pool.B [n, r, n_out]")
    n, _, r = A.shape
    N = B.shape[2]
    dt = _dtype_code(X)
    _need("X", X, (T, K), dtype, dev)
    if W is not None:
        _need("W", W, (K, N), dtype, dev)
    _need("pool.A", A, (n, K, r), dtype, dev)
    _need("pool.B", B, (n, r, N), dtype, dev)
    _need("pool.scale", pool.scale, (n,), torch.float32, dev)
    _need("ids", ids, (T,), torch.int32, dev)
    if Y is not None:
        _need("Y", Y, (T, N), dtype, dev)
    elif W is None:
        raise ValueError("without W the adapter terms are added to Y, which is missing")
    _on_gpu(X, ws)
    d = L.lora_multi_desc(T, K, N, r, n, dt, 0)
    with _on(stream):
        if Y is None:
            Y = torch.empty((T, N), dtype=X.dtype, device=dev)
        ws, ws_bytes = _ws_for(ws, multi_workspace_size(T, K, N, r, n, dt), dev)
    _call_on(X, stream, "lora_multi_fwd", C.byref(d), X.data_ptr(), _ptr(W), A.data_ptr(), B.data_ptr(),
             pool.scale.data_ptr(), ids.data_ptr(), Y.data_ptr(), ws.data_ptr(), ws_bytes)
    return Y


# ---------------------------------------------------------------------------
# Norms before and after a block
# ---------------------------------------------------------------------------

def _norm_call(R, Y, w_pre, w_post, gate, res_scale, branch_scale, eps, unit_offset):
    """The checked descriptor of a block norm over rows like R's."""
    T, H = _x2d("R", R)
    dt, shape, dtype, dev = _dtype_code(R), R.shape, R.dtype, R.device
    _need("R", R, shape, dtype, dev)
    if Y is not None:
        _need("Y", Y, shape, dtype, dev)
    kind, col = L.LORA_GATE_NONE, None
    if gate is not None:
        gs = gate.shape
        if gs == (H,):
            kind, col = L.LORA_GATE_COL, gate
        elif gs == (T, 1):
            kind = L.LORA_GATE_ROW
        elif gs == shape:
            kind = L.LORA_GATE_ELEM
        else:
            raise ValueError(f"gate has shape {tuple(gs)}, expected ({H},), ({T}, 1) or ({T}, {H})")
        if col is None:
            _need("gate", gate, gs, dtype, dev)
    first = w_pre if w_pre is not None else w_post if w_post is not None else col
    if first is not None:
        pd = first.dtype
        if pd != dtype:
            torch = _torch()
            if dtype != torch.bfloat16 or pd != torch.float32:
                raise ValueError(f"parameters in {pd} with activations in {dtype} are not supported")
            dt = L.LORA_BF16_F32LORA
        if w_pre is not None:
            _need("w_pre", w_pre, (H,), pd, dev)
        if w_post is not None:
            _need("w_post", w_post, (H,), pd, dev)
        if col is not None:
            _need("gate", col, (H,), pd, dev)
    return L.lora_norm_desc(T, H, eps, res_scale, branch_scale, int(unit_offset), kind, dt, 0)


@functools.lru_cache(maxsize=1024)
def block_norm_workspace_size(T, H, dtype=L.LORA_BF16):
    """Bytes of the backward's workspace (the forward takes none)."""
    d = L.lora_norm_desc(T, H, 0.0, 1.0, 1.0, 0, L.LORA_GATE_NONE, dtype, 0)
    b = C.c_size_t()
    L.call("lora_block_norm_workspace_size", C.byref(d), C.byref(b))
    return b.value


def block_norm_fwd(R, Y=None, *, w_pre=None, w_post=None, gate=None, res_scale=1.0, branch_scale=1.0, eps=1e-6,
                   unit_offset=False, R_out=None, X=None, stream=None):
    """Residual, gate and norms around a block with residual R and output Y, both [T, H]:

        p = norm(Y) w_post   (Y itself without w_post)
        R_out = res_scale R + branch_scale gate p
        X = norm(R_out) w_pre

    norm(v) = v / sqrt(mean(v^2) + eps) per row; unit_offset multiplies by 1 + w instead of w.
    gate: one value per column [H], per row [T, 1] or per element [T, H].
    Returns (R_out, X): X is None without w_pre; without Y (the first norm of a model) X = norm(R) w_pre and
    R_out is R.  R_out=R adds in place."""
    torch = _torch()
    d = _norm_call(R, Y, w_pre, w_post, gate, res_scale, branch_scale, eps, unit_offset)
    if Y is None and R_out is not None and R_out is not R:
        raise ValueError("R_out is written only when Y is given")
    if w_pre is None and X is not None:
        raise ValueError("X is written only when w_pre is given")
    if Y is not None and R_out is not None:
        _need("R_out", R_out, R.shape, R.dtype, R.device)
    if X is not None:
        _need("X", X, R.shape, R.dtype, R.device)
    _on_gpu(R)
    with _on(stream):
        if Y is not None and R_out is None:
            R_out = torch.empty_like(R)
        if w_pre is not None and X is None:
            X = torch.empty_like(R)
    _call_on(R, stream, "lora_block_norm_fwd", C.byref(d), _ptr(R), _ptr(Y), _ptr(gate), _ptr(w_post), _ptr(w_pre),
             None if Y is None else _ptr(R_out), _ptr(X))
    return (R if Y is None else R_out), X


def block_norm_bwd(dR_out, dX, R_out, Y=None, *, w_pre=None, w_post=None, gate=None, res_scale=1.0, branch_scale=1.0,
                   eps=1e-6, unit_offset=False, dR=None, dY=None, grads=None, ws=None, stream=None):
    """Gradients of block_norm_fwd, from those of its outputs (dR_out may be None: zero; dX exactly when the
    forward had w_pre), its R_out and its Y.  Returns (dR, dY, grads): grads holds "w_pre", "w_post" and "gate"
    for those the forward had, each of its parameter's shape and dtype; dY is None without Y.  dR and dY may be
    given, and may be dR_out, dX, R_out or Y themselves."""
    empty_like = _torch().empty_like
    d = _norm_call(R_out, Y, w_pre, w_post, gate, res_scale, branch_scale, eps, unit_offset)
    shape, dtype, dev = R_out.shape, R_out.dtype, R_out.device
    if w_pre is not None:
        _need("dX", dX, shape, dtype, dev)
    elif dX is not None:
        raise ValueError("dX needs w_pre")
    if dR_out is not None:
        _need("dR_out", dR_out, shape, dtype, dev)
    if dR is not None:
        _need("dR", dR, shape, dtype, dev)
    if dY is not None:
        _need("dY", dY, shape, dtype, dev)
        if Y is None:
            raise ValueError("dY needs Y")
    params = (("w_pre", w_pre), ("w_post", w_post), ("gate", gate))
    if grads is not None:
        for k, p in params:
            if p is not None:
                _need(f"grads[{k!r}]", grads.get(k), p.shape, p.dtype, dev)
    _on_gpu(R_out, ws)
    with _on(stream):
        if dR is None:
            dR = empty_like(R_out)
        if dY is None and Y is not None:
            dY = empty_like(Y)
        if grads is None:
            grads = {k: empty_like(p) for k, p in params if p is not None}
        ws, ws_bytes = _ws_for(ws, block_norm_workspace_size(d.T, d.H, d.dtype), dev)
    gr = L.lora_norm_grads(*[None if p is None else grads[k].data_ptr() for k, p in reversed(params)])
    _call_on(R_out, stream, "lora_block_norm_bwd", C.byref(d), _ptr(dR_out), _ptr(dX), R_out.data_ptr(), _ptr(Y),
             _ptr(gate), _ptr(w_post), _ptr(w_pre), dR.data_ptr(), _ptr(dY), C.byref(gr), ws.data_ptr(), ws_bytes)
    return dR, dY, grads


# ---------------------------------------------------------------------------
# Orthogonalised adapter updates
# ---------------------------------------------------------------------------

NS_COEFFS = (3.4445, -4.7750, 2.0315)


def _stacks(name, ts, like=None, dtype=None):
    """ts as a list of dense [rows, cols] or [count, rows, cols] tensors; with ``like``, of its shapes and device."""
    torch = _torch()
    ts = [ts] if torch.is_tensor(ts) else list(ts)
    if like is not None and len(ts) != len(like):
        raise ValueError(f"{name} holds {len(ts)} tensors, expected {len(like)}")
    for i, t in enumerate(ts):
        if t.dim() not in (2, 3):
            raise ValueError(f"{name}[{i}] must be [rows, cols] or [count, rows, cols], got shape {tuple(t.shape)}")
        _need(f"{name}[{i}]", t, (t if like is None else like[i]).shape, dtype or ts[0].dtype,
              (ts if like is None else like)[0].device)
    return ts


def _orth_mats(P, G, M, scale):
    mats = (L.lora_orth_mat * max(len(G), 1))()
    for m, p, g, s, k in zip(mats, P, G, M or [None] * len(G), scale):
        shape = g.shape
        m.G, m.M, m.P = g.data_ptr(), None if s is None else s.data_ptr(), p.data_ptr()
        m.count, m.rows, m.cols = (1, *shape) if len(shape) == 2 else shape
        m.scale = k
    return mats


def _orth_desc(n, steps, coeffs, eps, dtype):
    a, b, c = coeffs
    return L.lora_orth_desc(n, steps, a, b, c, eps, dtype, 0)


def _orth_ws(desc, mats):
    n = C.c_size_t()
    L.call("lora_orth_workspace_size", C.byref(desc), mats, C.byref(n))
    return n.value


def orth_workspace_size(mats):
    """Bytes of workspace of orthogonalize or muon_step for these matrices."""
    G = _stacks("mats", mats)
    if not G:
        return 0
    return _orth_ws(_orth_desc(len(G), 1, NS_COEFFS, 0.0, _dtype_code(G[0])), _orth_mats(G, G, None, [1.0] * len(G)))


def orthogonalize(mats, *, steps=5, coeffs=NS_COEFFS, eps=1e-7, out=None, ws=None, stream=None):
    """Newton-Schulz steps X <- a X + (b S + c S S) X, S = X X^T, from X = G / (|G| + eps), for every matrix of
    ``mats``: one tensor or a list of them, each [rows, cols] or a stack [count, rows, cols] with one side at
    most 64 (adapters or their gradients), bf16 or fp32.  Returns the same structure; ``out`` (or mats itself)
    receives the results.  |a|^steps may not exceed 2^22 (12 steps of the default coefficients), where the rounding
    of fp64 would reach the result."""
    torch = _torch()
    one = torch.is_tensor(mats)
    G = _stacks("mats", mats)
    if not G:
        return []
    desc = _orth_desc(len(G), steps, coeffs, eps, _dtype_code(G[0]))
    P = _stacks("out", out, G, G[0].dtype) if out is not None else None
    _on_gpu(G[0], ws)
    with _on(stream):
        if P is None:
            P = [torch.empty_like(g) for g in G]
        table = _orth_mats(P, G, None, [1.0] * len(G))
        if ws is None:
            ws = _ws(_orth_ws(desc, table), G[0].device)
    _call_on(G[0], stream, "lora_orthogonalize", C.byref(desc), table, _ptr(ws), _nbytes(ws, G[0].device))
    return P[0] if one else P


def muon_step(params, grads, moms, *, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=None, steps=5,
              coeffs=NS_COEFFS, eps=1e-7, ws=None, stream=None):
    """One optimizer step with orthogonalised updates, in place on params and moms:

        M <- momentum M + G;   U = G + momentum M (nesterov) or M
        P <- (1 - lr weight_decay) P - lr scale orthogonalize(U)

    params, grads (one dtype, bf16 or fp32) and moms (fp32) are tensors or lists as orthogonalize takes them.
    scale: a factor per entry of the list, one for all, or None: sqrt(max(1, cols / rows)), which for W [n_in,
    n_out] layouts gives updates of the same effect whatever the shape.
    Matrices of one shape are best kept as one stack [count, rows, cols]: a call takes three launches for every 24
    entries of the list whose short sides r have the same ceil(r / 16) (448 matrices of rank 16: 240 us in five
    stacks, 1250 us one by one).  |a|^steps is limited as in orthogonalize."""
    P = _stacks("params", params)
    if not P:
        return
    G = _stacks("grads", grads, P, P[0].dtype)
    M = _stacks("moms", moms, P, _torch().float32)
    if scale is None:
        scale = [max(1.0, p.shape[-1] / p.shape[-2]) ** 0.5 for p in P]
    elif isinstance(scale, (int, float)):
        scale = [scale] * len(P)
    elif len(scale) != len(P):
        raise ValueError(f"scale holds {len(scale)} values, expected {len(P)}")
    desc = L.lora_muon_desc(_orth_desc(len(P), steps, coeffs, eps, _dtype_code(P[0])), lr, momentum, weight_decay,
                            int(nesterov), 0)
    _on_gpu(P[0], ws)
    table = _orth_mats(P, G, M, scale)
    if ws is None:
        with _on(stream):
            ws = _ws(_orth_ws(desc.orth, table), P[0].device)
    _call_on(P[0], stream, "lora_muon_step", C.byref(desc), table, _ptr(ws), _nbytes(ws, P[0].device))


# ---------------------------------------------------------------------------
# NF4
# ---------------------------------------------------------------------------

def nf4_codebook():
    buf = (C.c_float * 16)()
    L.load().lora_nf4_codebook(buf)
    return list(buf)


def nf4_quantize(W, *, stream=None) -> NF4Weight:
    """Quantize a device weight W [rows, cols] (fp32 or bf16) to NF4 on the GPU."""
    torch = _torch()
    rows, cols = _x2d("W", W)
    if not W.is_contiguous():
        raise ValueError("W is not contiguous (the library takes dense row-major buffers)")
    _dtype_code(W)
    _on_gpu(W)
    n = rows * cols
    nbytes = C.c_size_t()
    L.call("lora_nf4_quantize_workspace_size", rows, cols, C.byref(nbytes))
    dev = W.device
    with _on(stream):
        w = NF4Weight(codes=torch.empty(n // 2, dtype=torch.uint8, device=dev),
                      q8=torch.empty(n // 64, dtype=torch.int8, device=dev),
                      s2=torch.empty(n // 16384, dtype=torch.float32, device=dev),
                      mu=torch.empty(1, dtype=torch.float32, device=dev), rows=rows, cols=cols)
        ws = _ws(nbytes.value, dev)
    L.call("lora_nf4_quantize", _ptr(W), rows, cols, _dtype_code(W), _ptr(w.codes), _ptr(w.q8), _ptr(w.s2),
           _ptr(w.mu), _ptr(ws), _nbytes(ws, dev), _stream(stream))
    return w


def nf4_dequant(w: NF4Weight, dtype=None, *, out=None, stream=None):
    torch = _torch()
    dtype = torch.bfloat16 if dtype is None else dtype
    _check_nf4("w", w, w.codes.device)
    if out is not None:
        _need("out", out, (w.rows, w.cols), dtype, w.codes.device)
    _on_gpu(w.codes)
    with _on(stream):
        if out is None:
            out = torch.empty((w.rows, w.cols), dtype=dtype, device=w.codes.device)
    s = w.c_struct()
    L.call("lora_nf4_dequant", C.byref(s), _ptr(out), _dtype_code(out), _stream(stream))
    return out


def nf4_unpack_codes(w: NF4Weight, *, stream=None):
    torch = _torch()
    _check_nf4("w", w, w.codes.device)
    _on_gpu(w.codes)
    with _on(stream):
        out = torch.empty(w.rows * w.cols, dtype=torch.uint8, device=w.codes.device)
    s = w.c_struct()
    L.call("lora_nf4_unpack_codes", C.byref(s), _ptr(out), _stream(stream))
    return out


def nf4_gemm(X, w: NF4Weight, A=None, B=None, scale=0.0, trans=False, *, Y=None, ws=None, stream=None):
    """trans=False: Y = X deq(W) + s (X A) B;  trans=True: Y = X deq(W)^T + s (X B^T) A^T."""
    torch = _torch()
    T, width = _x2d("X", X)
    k_in, n_out = (w.cols, w.rows) if trans else (w.rows, w.cols)
    if X.dtype != torch.bfloat16:
        raise ValueError(f"X has dtype {X.dtype}; the NF4 GEMM computes in bf16")
    _need("X", X, (T, k_in), torch.bfloat16, X.device)
    _check_nf4("w", w, X.device)
    if (A is None) != (B is None):
        raise ValueError("A and B must both be given or both be None")
    r = 0 if A is None else A.shape[1]
    if A is not None:
        _need("A", A, (w.rows, r), torch.bfloat16, X.device)
        _need("B", B, (r, w.cols), torch.bfloat16, X.device)
    if Y is not None:
        _need("Y", Y, (T, n_out), torch.bfloat16, X.device)
    _on_gpu(X, ws)
    nbytes = C.c_size_t()
    L.call("lora_nf4_gemm_workspace_size", T, w.rows, w.cols, r, int(trans), C.byref(nbytes))
    with _on(stream):
        if Y is None:
            Y = torch.empty((T, n_out), dtype=X.dtype, device=X.device)
        if ws is None:
            ws = _ws(nbytes.value, X.device)
    s = w.c_struct()
    L.call("lora_nf4_gemm", T, int(trans), _ptr(X), C.byref(s), _ptr(A), _ptr(B), r, float(scale), _ptr(Y),
           _ptr(ws), _nbytes(ws, X.device), _stream(stream))
    return Y


# ---------------------------------------------------------------------------
# Kernel timing
# ---------------------------------------------------------------------------

def trace_begin(prefix: str = "") -> None:
    """Record HIP-event durations of the library's launches (optionally only
    kernel families whose name starts with ``prefix``)."""
    L.call("lora_trace_begin", prefix.encode() if prefix else None)


def trace_end() -> dict:
    """Stop recording; returns {family: (launches, total_ms)}."""
    buf = (L.lora_trace_entry * 64)()
    n = C.c_int32()
    L.call("lora_trace_end", buf, 64, C.byref(n))
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(min(n.value, 64))}
