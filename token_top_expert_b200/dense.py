"""The dense MoE block for prompts and the operators it is made of: argument marshalling over
include/msb_dense.h, nothing else.

All calls are asynchronous on `stream` (default: torch's current stream) and launch on the
current device.  Outputs and scratch are allocated when not given; with a raw stream handle
pass them.
"""
from __future__ import annotations

import ctypes
import dataclasses

from . import _lib
from ._lib import MsbGroupWeights
from .block import Dims, PackedLayer, _act, _check, _ptr, _stream, _temporaries_on

_TYPES = None


def _type(t, what: str) -> int:
    global _TYPES
    if _TYPES is None:
        import torch
        _TYPES = {torch.bfloat16: _lib.MSB_BF16, torch.float32: _lib.MSB_F32}
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError("%s must be bf16 or float32, got %s" % (what, t.dtype))
    return code


def _here(lead, *others):
    """Every tensor on `lead`'s device, which is the current one."""
    dev = lead.device
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors, got one on %s" % dev)
    import torch
    if dev.index != torch.cuda.current_device():
        raise ValueError("the tensors are on %s but the current device is cuda:%d (the library "
                         "launches on the current device)" % (dev, torch.cuda.current_device()))
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError("tensors on %s and %s" % (dev, t.device))


def _rows2d(t, what: str) -> int:
    """Pitch in elements of a 2-d tensor whose last dimension is contiguous."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1 and t.shape[0] > 0):
        raise ValueError("%s must be 2-d with a contiguous last dimension, got %s strides %s"
                         % (what, tuple(t.shape), t.stride()))
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _ints(t, numel: int, what: str):
    if t is not None:
        import torch
        if t.dtype != torch.int32 or t.numel() < numel or not t.is_contiguous():
            raise ValueError("%s must be a contiguous int32 tensor of %d elements, got %s %s"
                             % (what, numel, t.dtype, tuple(t.shape)))


def dense_check(stream=None):
    """Raise MsbError if a kernel of this module's calls on the current device was flagged
    since the last check (synchronises the stream)."""
    _check(_lib.load().msb_dense_check(_stream(stream)), "dense kernel")


# ------------------------------------------------------------------ routing

@dataclasses.dataclass
class Routing:
    """A batch's routing (see msb_route in include/msb_dense.h): ids, weights, pos are
    [tokens][top_e], rows [tokens * top_e], offsets [experts + 1]."""
    ids: object
    weights: object
    offsets: object
    rows: object
    pos: object

    @classmethod
    def empty(cls, tokens: int, experts: int, top_e: int, device="cuda") -> "Routing":
        import torch
        i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=device)  # noqa: E731
        return cls(i32(tokens, top_e), torch.empty((tokens, top_e), dtype=torch.float32, device=device),
                   i32(experts + 1), i32(tokens * top_e), i32(tokens, top_e))


def route(logits, top_e: int, renorm: bool = True, mask=None, out: Routing | None = None,
          workspace=None, stream=None) -> Routing:
    """Top-K experts of each token from its router logits (bf16 or float32 [tokens][experts]),
    their weights, and the pairs sorted by expert.  mask: bool or uint8 [tokens], 0 for tokens
    that take no part.  workspace: uint8 scratch of msb_route_workspace_size bytes."""
    import torch
    lib = _lib.load()
    ld = _rows2d(logits, "logits")
    T, E = logits.shape
    new = []
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or tuple(mask.shape) != (T,)
                             or not mask.is_contiguous()):
        raise ValueError("mask must be a contiguous bool or uint8 tensor of %d tokens" % T)
    if not 1 <= top_e <= E:
        raise ValueError("top_e must lie in 1..%d" % E)
    if out is None:
        out = Routing.empty(T, E, top_e, logits.device)
        new += [out.ids, out.weights, out.offsets, out.rows, out.pos]
    else:
        for name, n in (("ids", T * top_e), ("offsets", E + 1), ("rows", T * top_e), ("pos", T * top_e)):
            _ints(getattr(out, name), n, "out." + name)
        if out.weights.dtype != torch.float32 or out.weights.numel() < T * top_e or not out.weights.is_contiguous():
            raise ValueError("out.weights must be a contiguous float32 tensor of %d elements" % (T * top_e))
    if workspace is None:
        workspace = torch.empty(max(1, lib.msb_route_workspace_size(T, E)), dtype=torch.uint8,
                                device=logits.device)
        new.append(workspace)
    _here(logits, mask, out.ids, out.weights, out.offsets, out.rows, out.pos, workspace)
    _temporaries_on(stream, new)
    _check(lib.msb_route(logits.data_ptr(), _type(logits, "logits"), ld, _ptr(mask), T, E, top_e,
                         1 if renorm else 0, out.ids.data_ptr(), out.weights.data_ptr(),
                         out.offsets.data_ptr(), out.rows.data_ptr(), out.pos.data_ptr(),
                         workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                         _stream(stream)), "msb_route")
    return out


# ------------------------------------------------------------------ grouped products

def _weights(w, dtype, parts: bool):
    """(msb_group_weights, groups, n, k) of a [groups][n][k] or [groups][2][n][k] tensor (one
    group: without the leading dimension), any strides the C ABI takes."""
    if w.dtype != dtype:
        raise ValueError("the weights must be %s, got %s" % (dtype, w.dtype))
    dims = 3 if parts else 2
    if w.dim() not in (dims, dims + 1):
        raise ValueError("weights of shape %s: expected %s" % (tuple(w.shape), (
            "[groups][2][n][k]" if parts else "[groups][n][k]")))
    shape, stride = tuple(w.shape), w.stride()
    if w.dim() == dims:
        shape, stride = (1,) + shape, (0,) + stride
    if parts and shape[1] != 2:
        raise ValueError("weights of shape %s: the gate and up parts are dimension -3" % (tuple(w.shape),))
    sn, sk = stride[-2:]
    n, k = shape[-2:]
    if k == 1 and sn != 1:
        sk = 1
    return (MsbGroupWeights(w.data_ptr(), stride[0], stride[1] if parts else 0, sn, sk), shape[0], n, k)


def _product(fn_name, x, w, offsets, rows, out, out_dtype, stream, parts, scales=None):
    import torch
    i8 = scales is not None
    gw, groups, n, k = _weights(w, torch.int8 if i8 else torch.bfloat16, parts)
    if x.dtype != w.dtype:
        raise ValueError("x must be %s, got %s" % (w.dtype, x.dtype))
    ldx = _rows2d(x, "x")
    if x.shape[1] != k:
        raise ValueError("x has %d columns, the weights %d" % (x.shape[1], k))
    if offsets is None and groups != 1:
        raise ValueError("offsets are required with %d groups" % groups)
    _ints(offsets, groups + 1, "offsets")
    r = x.shape[0] if rows is None else rows.numel()
    _ints(rows, r, "rows")
    new = []
    if out is None:
        out = torch.empty((r, n), dtype=out_dtype or torch.bfloat16, device=x.device)
        new = [out]
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
    ldo = _rows2d(out, "out")
    # out may have rows behind the last group's; without offsets every row is computed
    if out.shape[1] != n or out.shape[0] < r or (offsets is None and out.shape[0] != r):
        raise ValueError("out is %s, this call needs [%d][%d]" % (tuple(out.shape), r, n))
    code = _type(out, "out")
    if parts and code != _lib.MSB_BF16:
        raise ValueError("SwiGLU products are bf16")
    extra = ()
    if i8:
        q_scale, w_scale = scales
        want = (groups, 2, n) if parts else (groups, n)
        if q_scale.dtype != torch.float32 or q_scale.numel() != x.shape[0] or not q_scale.is_contiguous():
            raise ValueError("the rows' scales must be a contiguous float32 tensor of %d" % x.shape[0])
        if (w_scale.dtype != torch.float32 or not w_scale.is_contiguous() or
                tuple(w_scale.shape) != (want if w.dim() == len(want) + 1 else want[1:])):
            raise ValueError("the weights' scales must be contiguous float32 %s" % (want,))
        _here(x, w, offsets, rows, out, q_scale, w_scale)
        extra = (q_scale, w_scale)
    else:
        _here(x, w, offsets, rows, out)
    _temporaries_on(stream, new)
    args = [x.data_ptr(), ldx]
    if i8:
        args.append(extra[0].data_ptr())
    args += [x.shape[0], _ptr(rows), _ptr(offsets), groups, r, ctypes.byref(gw)]
    if i8:
        args.append(extra[1].data_ptr())
    args += [n, k, out.data_ptr()]
    if not parts:
        args.append(code)
    _check(getattr(_lib.load(), fn_name)(*args, ldo, _stream(stream)), fn_name)
    return out


def grouped_matmul(x, w, offsets=None, rows=None, out=None, out_dtype=None, stream=None):
    """out[p] = x[row(p)] @ w[e].T for the rows p of group e (offsets[e] <= p < offsets[e + 1]).
    x: bf16 [rows][k]; w: bf16 [groups][n][k] view with n or k contiguous (or [n][k]: one
    group); offsets: int32 [groups + 1]; rows: int32, the row of x of each output row (default:
    itself); out: bf16 or float32 [rows][n], rows of no group are left as they are."""
    return _product("msb_grouped_matmul", x, w, offsets, rows, out, out_dtype, stream, False)


def grouped_swiglu(x, w, offsets=None, rows=None, out=None, stream=None):
    """silu(x @ w[e][0].T) * (x @ w[e][1].T) by groups, bf16; w: bf16 [groups][2][n][k]."""
    return _product("msb_grouped_swiglu", x, w, offsets, rows, out, None, stream, True)


# ------------------------------------------------------------------ 8-bit integers

def quantize_int8(x, out=None, scale=None, stream=None):
    """Rows of x (bf16 or float32 [rows][k]) as 8-bit integers with one scale each: returns
    (q int8 [rows][k] on a pitch of whole 16 bytes, scale float32 [rows])."""
    import torch
    ldx = _rows2d(x, "x")
    R, k = x.shape
    new = []
    if out is None:
        buf = torch.empty((R, (k + 15) // 16 * 16), dtype=torch.int8, device=x.device)
        out = buf if buf.shape[1] == k else buf[:, :k]
        new.append(buf)
    if scale is None:
        scale = torch.empty(R, dtype=torch.float32, device=x.device)
        new.append(scale)
    if out.dtype != torch.int8 or tuple(out.shape) != (R, k):
        raise ValueError("out must be int8 [%d][%d]" % (R, k))
    if scale.dtype != torch.float32 or scale.numel() != R or not scale.is_contiguous():
        raise ValueError("scale must be a contiguous float32 tensor of %d" % R)
    ldq = _rows2d(out, "out")
    _here(x, out, scale)
    _temporaries_on(stream, new)
    _check(_lib.load().msb_int8_quantize(x.data_ptr(), _type(x, "x"), ldx, R, k, out.data_ptr(), ldq,
                                         scale.data_ptr(), _stream(stream)), "msb_int8_quantize")
    return out, scale


def matmul_int8(q, q_scale, w, w_scale, offsets=None, rows=None, out=None, out_dtype=None,
                swiglu: bool = False, stream=None):
    """grouped_matmul (or grouped_swiglu) on 8-bit integers: q int8 [rows][k] with q_scale
    float32 [rows], w int8 like the bf16 weights (k contiguous) with w_scale float32 of w's
    shape without k."""
    return _product("msb_int8_swiglu" if swiglu else "msb_int8_matmul", q, w, offsets, rows, out,
                    None if swiglu else out_dtype, stream, swiglu, (q_scale, w_scale))


def linear_int8(x, w, w_scale, offsets=None, rows=None, out=None, out_dtype=None, stream=None):
    """x (bf16 or float32) quantised row by row and multiplied in 8-bit integers."""
    q, s = quantize_int8(x, stream=stream)
    return matmul_int8(q, s, w, w_scale, offsets, rows, out, out_dtype, False, stream)


def swiglu_int8(x, w, w_scale, offsets=None, rows=None, out=None, stream=None):
    """linear_int8 for gate and up ([groups][2][n][k]) with SwiGLU."""
    q, s = quantize_int8(x, stream=stream)
    return matmul_int8(q, s, w, w_scale, offsets, rows, out, None, True, stream)


# ------------------------------------------------------------------ combine, norms

def combine(y, routing: Routing, out=None, stream=None):
    """out[t] = sum_k weights[t][k] * y[pos[t][k]] (bf16 [tokens][d]); y bf16 or float32."""
    import torch
    ldy = _rows2d(y, "y")
    if routing.pos.dim() != 2 or routing.weights.shape != routing.pos.shape:
        raise ValueError("routing.pos and routing.weights must be [tokens][top_e]")
    T, K = routing.pos.shape
    _ints(routing.pos, T * K, "routing.pos")
    if routing.weights.dtype != torch.float32 or not routing.weights.is_contiguous():
        raise ValueError("routing.weights must be contiguous float32")
    new = []
    if out is None:
        out = torch.empty((T, y.shape[1]), dtype=torch.bfloat16, device=y.device)
        new = [out]
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (T, y.shape[1]):
        raise ValueError("out must be bf16 [%d][%d]" % (T, y.shape[1]))
    ldo = _rows2d(out, "out")
    _here(y, routing.pos, routing.weights, out)
    _temporaries_on(stream, new)
    _check(_lib.load().msb_combine(y.data_ptr(), _type(y, "y"), ldy, y.shape[0], routing.pos.data_ptr(),
                                   routing.weights.data_ptr(), T, K, y.shape[1], out.data_ptr(), ldo,
                                   _stream(stream)), "msb_combine")
    return out


def block_norm(h, y=None, x=None, h_out=None, pre_weight=None, post_norm: bool = False,
               post_weight=None, gate=None, skip_scale: float = 1.0, residual_scale: float = 1.0,
               eps: float = 1e-6, stream=None):
    """The glue around a block (msb_block_norm): h' = skip_scale h + residual_scale gate b with
    b = y, or rms-normed y times post_weight; x = rms-normed h' times pre_weight.  h, y: bf16 or
    float32 [rows][d]; gate: [d], or 2-d and broadcastable to [rows][d]; x: bf16 output
    (allocated when None); h_out: where h' goes (default: h itself).  Returns (h', x)."""
    import torch
    ldh = _rows2d(h, "h")
    R, d = h.shape
    new = []
    if x is None:
        x = torch.empty((R, d), dtype=torch.bfloat16, device=h.device)
        new = [x]
    if h_out is None:
        h_out = h
    for name, t in (("y", y), ("x", x), ("h_out", h_out)):
        if t is not None and t.shape != h.shape:
            raise ValueError("%s must be shaped like h" % name)
    if x.dtype != torch.bfloat16 or h_out.dtype != h.dtype:
        raise ValueError("x must be bf16 and h_out of h's type")
    wtype = 0
    for name, t in (("pre_weight", pre_weight), ("post_weight", post_weight)):
        if t is not None:
            if tuple(t.shape) != (d,) or not t.is_contiguous():
                raise ValueError("%s must be a contiguous tensor of %d elements" % (name, d))
            wtype = _type(t, name)
    if pre_weight is not None and post_weight is not None and pre_weight.dtype != post_weight.dtype:
        raise ValueError("pre_weight and post_weight must have one type")
    gtype = grow = gcol = 0
    if gate is not None:
        gtype = _type(gate, "gate")
        if gate.dim() == 1 and gate.shape[0] == d:
            gcol = gate.stride(0)
        elif gate.dim() == 2 and gate.shape[0] in (1, R) and gate.shape[1] in (1, d):
            grow = gate.stride(0) if gate.shape[0] > 1 else 0
            gcol = gate.stride(1) if gate.shape[1] > 1 else 0
        else:
            raise ValueError("gate must be [d] or broadcastable [rows][d], got %s" % (tuple(gate.shape),))
    _here(h, y, x, h_out, pre_weight, post_weight, gate)
    _temporaries_on(stream, new)
    _check(_lib.load().msb_block_norm(
        h.data_ptr(), _type(h, "h"), ldh, _ptr(y), 0 if y is None else _type(y, "y"),
        0 if y is None else _rows2d(y, "y"), _ptr(pre_weight), _ptr(post_weight), wtype,
        1 if post_norm else 0, _ptr(gate), gtype, grow, gcol, skip_scale, residual_scale, eps,
        h_out.data_ptr(), _rows2d(h_out, "h_out"), x.data_ptr(), _rows2d(x, "x"), R, d,
        _stream(stream)), "msb_block_norm")
    return h_out, x


# ------------------------------------------------------------------ the dense block

class Int8Layer:
    """One MoE layer's experts in 8-bit integers with a scale for every output channel:
    gate_up int8 [E][2][I][d], down int8 [E][d][Ipad], scales float32 [E][2][I] and [E][d];
    router_t as in PackedLayer."""

    def __init__(self, dims: Dims, gate_up, gate_up_scale, down, down_scale, router_t):
        import torch
        d, I, E = dims.d, dims.inter, dims.experts
        want = (("gate_up", gate_up, (E, 2, I, d), torch.int8),
                ("gate_up_scale", gate_up_scale, (E, 2, I), torch.float32),
                ("down", down, (E, d, dims.ipad), torch.int8),
                ("down_scale", down_scale, (E, d), torch.float32))
        for name, t, shape, dtype in want:
            if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous() or t.device != gate_up.device:
                raise ValueError("%s: expected contiguous %s %s, got %s %s" % (name, dtype, shape, t.dtype, tuple(t.shape)))
        if (router_t.numel() != E * d or router_t.element_size() != 2 or not router_t.is_contiguous()
                or router_t.device != gate_up.device):
            raise ValueError("router_t: expected %d contiguous 2-byte elements" % (E * d))
        self.dims, self.gate_up, self.gate_up_scale = dims, gate_up, gate_up_scale
        self.down, self.down_scale, self.router_t = down, down_scale, router_t

    @classmethod
    def from_packed(cls, layer: PackedLayer) -> "Int8Layer":
        """Quantise a bf16 layer on its device: each gate, up and down row (output channel) with
        its own scale."""
        import torch
        if layer.q4:
            raise ValueError("4-bit records: quantise the bf16 layer")
        dims = layer.dims
        d, I, E = dims.d, dims.inter, dims.experts
        rec = layer.records.view(torch.bfloat16).view(E, I, 3, d)
        gate_up = torch.empty((E, 2, I, d), dtype=torch.int8, device=rec.device)
        gs = torch.empty((E, 2, I), dtype=torch.float32, device=rec.device)
        down = torch.zeros((E, d, dims.ipad), dtype=torch.int8, device=rec.device)
        ds = torch.empty((E, d), dtype=torch.float32, device=rec.device)
        for e in range(E):
            for p in range(2):
                quantize_int8(rec[e, :, p], gate_up[e, p], gs[e, p])
            quantize_int8(rec[e, :, 2].t().contiguous(), down[e][:, :I], ds[e])
        return cls(dims, gate_up, gs, down, ds, layer.router_t)


class DenseWorkspace:
    """Device scratch of moe_dense_block calls of up to `tokens` tokens."""

    def __init__(self, dims: Dims, tokens: int, int8: bool = False, device="cuda"):
        import torch
        n = _lib.load().msb_dense_workspace_size(ctypes.byref(dims.c()), tokens, 1 if int8 else 0)
        if n == 0:
            raise ValueError("invalid dims or tokens for a workspace")
        self.nbytes = n
        self.buf = torch.empty(n, dtype=torch.uint8, device=device)
        self.ptr = self.buf.data_ptr()


def moe_dense_block(x, layer, out=None, mask=None, workspace: DenseWorkspace | None = None, stream=None):
    """The dense MoE block (every channel of each routed expert, no compensation term) on any
    number of tokens: what moe_sparse_block computes with k = I and rank 0.  x: bf16
    [tokens][d]; layer: a bf16 PackedLayer or an Int8Layer; mask: bool or uint8 [tokens],
    tokens with 0 get zeros."""
    import torch
    dims = layer.dims
    _act(x, dims)
    int8 = isinstance(layer, Int8Layer)
    if not int8 and layer.q4:
        raise ValueError("4-bit records: use moe_sparse_block")
    T = x.shape[0]
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or tuple(mask.shape) != (T,)
                             or not mask.is_contiguous()):
        raise ValueError("mask must be a contiguous bool or uint8 tensor of %d tokens" % T)
    new = []
    if out is None:
        out = torch.empty_like(x)
        new.append(out)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor shaped like x")
    if workspace is None:
        workspace = DenseWorkspace(dims, T, int8, x.device)
        new.append(workspace.buf)
    _here(x, layer.router_t, out, mask, workspace.buf)
    _temporaries_on(stream, new)
    lib, cd = _lib.load(), dims.c()
    tail = (out.data_ptr(), ctypes.byref(cd), workspace.ptr, workspace.nbytes, _stream(stream))
    head = (x.data_ptr(), T, _ptr(mask), layer.router_t.data_ptr())
    if int8:
        rc = lib.moe_dense_block_int8(*head, layer.gate_up.data_ptr(), layer.gate_up_scale.data_ptr(),
                                      layer.down.data_ptr(), layer.down_scale.data_ptr(), *tail)
    else:
        rc = lib.moe_dense_block(*head, layer.records.data_ptr(), *tail)
    _check(rc, "moe_dense_block")
    return out
