"""The dense MoE block for prompts and the operators it is made of: argument marshalling over
include/msb_dense.h, nothing else.

All calls are asynchronous on `stream` (default: torch's current stream) and launch on the
current device.  Outputs and scratch are allocated when not given; with a raw stream handle
pass them.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools

from . import _lib
from ._lib import MsbGroupWeights
from .block import Dims, PackedLayer, _act, _check, _ptr, _stream, _temporaries_on

_raw = None  # torch's current stream of a device as a handle, without a Stream object


@functools.lru_cache(maxsize=256)
def _route_bytes(tokens: int, experts: int) -> int:
    return _lib.load().msb_route_workspace_size(tokens, experts)


@functools.lru_cache(maxsize=256)
def _linear_bytes(rows: int, k: int) -> int:
    return _lib.load().msb_int8_linear_workspace_size(rows, k)


def _types():
    import torch
    global _raw
    _raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    return {torch.bfloat16: _lib.MSB_BF16, torch.float32: _lib.MSB_F32}


_TYPES: dict = {}


def _type(t, what: str) -> int:
    if not _TYPES:
        _TYPES.update(_types())
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError("%s must be bf16 or float32, got %s" % (what, t.dtype))
    return code


def _here(lead, *others) -> int:
    """Every tensor on `lead`'s device, which is the current one; its index."""
    dev = lead.get_device()
    if dev < 0:
        raise ValueError("expected CUDA tensors, got one on %s" % lead.device)
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors on %s and %s" % (lead.device, t.device))
    import torch
    if dev != torch.cuda.current_device():
        raise ValueError("the tensors are on cuda:%d but the current device is cuda:%d (the library "
                         "launches on the current device)" % (dev, torch.cuda.current_device()))
    return dev


def _on(stream, dev: int, new) -> int:
    """The call's stream as a handle, ordered after the allocation of the buffers `new`."""
    if stream is None:
        if _raw is None:
            _TYPES.update(_types())
        return _raw(dev)
    _temporaries_on(stream, new)
    return _stream(stream)


def _rows2d(t, what: str) -> int:
    """Pitch in elements of a 2-d tensor whose last dimension is contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1 and shape[0] > 0):
        raise ValueError("%s must be 2-d with a contiguous last dimension, got %s strides %s"
                         % (what, tuple(shape), stride))
    return stride[0] if shape[0] > 1 else max(shape[1], 1)


def _ints(t, numel: int, what: str):
    import torch
    if t.dtype is not torch.int32 or t.numel() < numel or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of %d elements, got %s %s"
                         % (what, numel, t.dtype, tuple(t.shape)))


def _floats(t, shape, what: str):
    import torch
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous float32 tensor %s, got %s %s"
                         % (what, tuple(shape), t.dtype, tuple(t.shape)))


def _scratch(t):
    """(address, bytes) of a caller's workspace, whose bytes must lie in a row."""
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous, got strides %s" % (t.stride(),))
    return t.data_ptr(), t.numel() * t.element_size()


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
        return cls._in(_routing_buffer(tokens, experts, top_e, 0, device), tokens, experts, top_e)

    @classmethod
    def _in(cls, buf, tokens: int, experts: int, top_e: int) -> "Routing":
        import torch
        n, shape, stride, part = tokens * top_e, (tokens, top_e), (top_e, 1), buf.as_strided
        return cls(part(shape, stride, 0), part(shape, stride, n).view(torch.float32),
                   part((experts + 1,), (1,), 4 * n), part((n,), (1,), 3 * n), part(shape, stride, 2 * n))


def _routing_buffer(tokens, experts, top_e, scratch, device):
    """One allocation for a Routing (and `scratch` bytes behind it)."""
    import torch
    return torch.empty(4 * tokens * top_e + experts + 1 + (scratch + 3) // 4, dtype=torch.int32, device=device)


def _mask(mask, tokens: int):
    import torch
    if (mask.dtype not in (torch.bool, torch.uint8) or tuple(mask.shape) != (tokens,)
            or not mask.is_contiguous()):
        raise ValueError("mask must be a contiguous bool or uint8 tensor of %d tokens" % tokens)


def route(logits, top_e: int, renorm: bool = True, mask=None, out: Routing | None = None,
          workspace=None, stream=None) -> Routing:
    """Top-K experts of each token from its router logits (bf16 or float32 [tokens][experts]),
    their weights, and the pairs sorted by expert.  mask: bool or uint8 [tokens], 0 for tokens
    that take no part.  workspace: uint8 scratch of msb_route_workspace_size bytes."""
    lib = _lib.load()
    ld = _rows2d(logits, "logits")
    T, E = logits.shape
    code = _type(logits, "logits")
    if not 1 <= top_e <= E:
        raise ValueError("top_e must lie in 1..%d" % E)
    n = T * top_e
    need = _route_bytes(T, E)
    if mask is not None:
        _mask(mask, T)
    given = None if workspace is None else _scratch(workspace)
    new = []
    if out is None:
        buf = _routing_buffer(T, E, top_e, need if workspace is None else 0, logits.device)
        out = Routing._in(buf, T, E, top_e)
        new.append(buf)
        base = buf.data_ptr()
        at = (base, base + 4 * n, base + 16 * n, base + 12 * n, base + 8 * n)
        ws, nb = base + 4 * (4 * n + E + 1), need
        dev = _here(logits, mask, workspace)
    else:
        for name, k in (("ids", n), ("offsets", E + 1), ("rows", n), ("pos", n)):
            _ints(getattr(out, name), k, "out." + name)
        _floats(out.weights, (T, top_e), "out.weights")
        dev = _here(logits, mask, out.ids, out.weights, out.offsets, out.rows, out.pos, workspace)
        at = tuple(t.data_ptr() for t in (out.ids, out.weights, out.offsets, out.rows, out.pos))
        if workspace is None:
            import torch
            buf = torch.empty(max(1, need), dtype=torch.uint8, device=logits.device)
            new.append(buf)
            ws, nb = buf.data_ptr(), need
    if given:
        ws, nb = given
    rc = lib.msb_route(logits.data_ptr(), code, ld, _ptr(mask), T, E, top_e, 1 if renorm else 0, *at, ws, nb,
                       _on(stream, dev, new))
    if rc:
        _check(rc, "msb_route")
    return out


# ------------------------------------------------------------------ grouped products

def _weights(w, parts: bool):
    """(msb_group_weights, groups, n, k) of a [groups][n][k] or [groups][2][n][k] tensor (one
    group: without the leading dimension), any strides the C ABI takes."""
    shape, stride = w.shape, w.stride()
    dims = 3 if parts else 2
    if len(shape) == dims:
        shape, stride = (1, *shape), (0, *stride)
    if len(shape) != dims + 1 or (parts and shape[1] != 2):
        raise ValueError("weights of shape %s: expected %s" % (tuple(w.shape), (
            "[groups][2][n][k]" if parts else "[groups][n][k]")))
    n, k = shape[-2:]
    sn, sk = stride[-2:]
    if k == 1 and sn != 1:
        sk = 1
    return MsbGroupWeights(w.data_ptr(), stride[0], stride[1] if parts else 0, sn, sk), shape[0], n, k


def _product(what, x, w, offsets, rows, out, out_dtype, stream, parts, q_scale=None, w_scale=None, q=None,
             workspace=None):
    """One grouped product.  q: quantise x on the way (None: x is what is multiplied), in `workspace`."""
    import torch
    i8 = w_scale is not None
    gw, groups, n, k = _weights(w, parts)
    if w.dtype is not (torch.int8 if i8 else torch.bfloat16) or (q is None and x.dtype is not w.dtype):
        raise ValueError("x is %s and the weights %s" % (x.dtype, w.dtype))
    ldx = _rows2d(x, "x")
    R, cols = x.shape
    if cols != k:
        raise ValueError("x has %d columns, the weights %d" % (cols, k))
    if offsets is not None:
        _ints(offsets, groups + 1, "offsets")
    elif groups != 1:
        raise ValueError("offsets are required with %d groups" % groups)
    r = R
    if rows is not None:
        r = rows.numel()
        _ints(rows, r, "rows")
    new = []
    if out is None:
        out = torch.empty(r, n, dtype=out_dtype or torch.bfloat16, device=x.device)
        new.append(out)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise ValueError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
    ldo = _rows2d(out, "out")
    # out may have rows behind the last group's; without offsets every row is computed
    if out.shape[1] != n or out.shape[0] < r or (offsets is None and out.shape[0] != r):
        raise ValueError("out is %s, this call needs [%d][%d]" % (tuple(out.shape), r, n))
    code = _type(out, "out")
    if parts and code != _lib.MSB_BF16:
        raise ValueError("SwiGLU products are bf16")
    given = None if workspace is None else _scratch(workspace)
    dev = _here(x, w, offsets, rows, out, q_scale, w_scale, workspace)
    off, row, o = _ptr(offsets), _ptr(rows), out.data_ptr()
    lib = _lib.load()
    if not i8:
        fn = lib.msb_grouped_swiglu if parts else lib.msb_grouped_matmul
        rc = fn(x.data_ptr(), ldx, R, row, off, groups, r, gw, n, k, o, *(() if parts else (code,)), ldo,
                _on(stream, dev, new))
    else:
        want = (groups, 2, n) if parts else (groups, n)
        _floats(w_scale, want if w.dim() == len(want) + 1 else want[1:], "the weights' scales")
        if q is None:
            _floats(q_scale, (R,), "the rows' scales")
            fn = lib.msb_int8_swiglu if parts else lib.msb_int8_matmul
            rc = fn(x.data_ptr(), ldx, q_scale.data_ptr(), R, row, off, groups, r, gw, w_scale.data_ptr(), n, k, o,
                    *(() if parts else (code,)), ldo, _on(stream, dev, new))
        else:
            nb = _linear_bytes(R, k)
            if nb == 0:
                raise ValueError("x of %d rows of %d is beyond the library's limits" % (R, k))
            if workspace is None:
                ws = torch.empty(nb, dtype=torch.uint8, device=x.device)
                new.append(ws)
                given = ws.data_ptr(), nb
            rc = lib.msb_int8_linear(x.data_ptr(), _type(x, "x"), ldx, R, row, off, groups, r, gw,
                                     w_scale.data_ptr(), n, k, 1 if parts else 0, o, code, ldo, *given,
                                     _on(stream, dev, new))
    if rc:
        _check(rc, what)
    return out


def grouped_matmul(x, w, offsets=None, rows=None, out=None, out_dtype=None, stream=None):
    """out[p] = x[row(p)] @ w[e].T for the rows p of group e (offsets[e] <= p < offsets[e + 1]).
    x: bf16 [rows][k]; w: bf16 [groups][n][k] view with n or k contiguous (or [n][k]: one
    group); offsets: int32 [groups + 1]; rows: int32, the row of x of each output row (default:
    itself); out: bf16 or float32 [rows][n], rows of no group are left as they are."""
    return _product("grouped_matmul", x, w, offsets, rows, out, out_dtype, stream, False)


def grouped_swiglu(x, w, offsets=None, rows=None, out=None, stream=None):
    """silu(x @ w[e][0].T) * (x @ w[e][1].T) by groups, bf16; w: bf16 [groups][2][n][k]."""
    return _product("grouped_swiglu", x, w, offsets, rows, out, None, stream, True)


# ------------------------------------------------------------------ 8-bit integers

def quantize_int8(x, out=None, scale=None, stream=None):
    """Rows of x (bf16 or float32 [rows][k]) as 8-bit integers with one scale each: returns
    (q int8 [rows][k] on a pitch of whole 16 bytes, scale float32 [rows])."""
    import torch
    ldx = _rows2d(x, "x")
    R, k = x.shape
    new = []
    if out is None:
        pitch = (k + 15) // 16 * 16
        out = torch.empty(R, pitch, dtype=torch.int8, device=x.device)
        new.append(out)
        if pitch != k:
            out = out[:, :k]
    if scale is None:
        scale = torch.empty(R, dtype=torch.float32, device=x.device)
        new.append(scale)
    if out.dtype is not torch.int8 or out.shape != x.shape:
        raise ValueError("out must be int8 [%d][%d]" % (R, k))
    _floats(scale, (R,), "scale")
    ldq = _rows2d(out, "out")
    code = _type(x, "x")
    dev = _here(x, out, scale)
    rc = _lib.load().msb_int8_quantize(x.data_ptr(), code, ldx, R, k, out.data_ptr(), ldq, scale.data_ptr(),
                                       _on(stream, dev, new))
    if rc:
        _check(rc, "quantize_int8")
    return out, scale


def matmul_int8(q, q_scale, w, w_scale, offsets=None, rows=None, out=None, out_dtype=None,
                swiglu: bool = False, stream=None):
    """grouped_matmul (or grouped_swiglu) on 8-bit integers: q int8 [rows][k] with q_scale
    float32 [rows], w int8 like the bf16 weights (k contiguous) with w_scale float32 of w's
    shape without k.  SwiGLU products are bf16."""
    return _product("matmul_int8", q, w, offsets, rows, out, out_dtype, stream, swiglu, q_scale, w_scale)


def linear_int8(x, w, w_scale, offsets=None, rows=None, out=None, out_dtype=None, stream=None, workspace=None):
    """x (bf16 or float32) quantised row by row and multiplied in 8-bit integers.  workspace: uint8
    scratch of msb_int8_linear_workspace_size bytes."""
    return _product("linear_int8", x, w, offsets, rows, out, out_dtype, stream, False, None, w_scale, True, workspace)


def swiglu_int8(x, w, w_scale, offsets=None, rows=None, out=None, stream=None, workspace=None):
    """linear_int8 for gate and up ([groups][2][n][k]) with SwiGLU."""
    return _product("swiglu_int8", x, w, offsets, rows, out, None, stream, True, None, w_scale, True, workspace)


# ------------------------------------------------------------------ combine, norms

def combine(y, routing: Routing, out=None, stream=None):
    """out[t] = sum_k weights[t][k] * y[pos[t][k]] (bf16 [tokens][d]); y bf16 or float32."""
    import torch
    ldy = _rows2d(y, "y")
    pos, weights = routing.pos, routing.weights
    if pos.dim() != 2:
        raise ValueError("routing.pos must be [tokens][top_e]")
    T, K = pos.shape
    _ints(pos, T * K, "routing.pos")
    _floats(weights, (T, K), "routing.weights")
    d = y.shape[1]
    new = []
    if out is None:
        out = torch.empty(T, d, dtype=torch.bfloat16, device=y.device)
        new.append(out)
    elif out.dtype is not torch.bfloat16 or out.shape != (T, d):
        raise ValueError("out must be bf16 [%d][%d]" % (T, d))
    ldo = _rows2d(out, "out")
    code = _type(y, "y")
    dev = _here(y, pos, weights, out)
    rc = _lib.load().msb_combine(y.data_ptr(), code, ldy, y.shape[0], pos.data_ptr(), weights.data_ptr(), T, K, d,
                                 out.data_ptr(), ldo, _on(stream, dev, new))
    if rc:
        _check(rc, "combine")
    return out


def _norm_weight(t, d: int, what: str):
    if t.shape != (d,) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of %d elements" % (what, d))
    return _type(t, what)


def block_norm(h, y=None, x=None, h_out=None, pre_weight=None, post_norm: bool = False,
               post_weight=None, gate=None, skip_scale: float = 1.0, residual_scale: float = 1.0,
               eps: float = 1e-6, stream=None):
    """The glue around a block (msb_block_norm): h' = skip_scale h + residual_scale gate b with
    b = y, or rms-normed y times post_weight; x = rms-normed h' times pre_weight.  h, y: bf16 or
    float32 [rows][d]; gate: [d], or 2-d and broadcastable to [rows][d]; x: bf16 output
    (allocated when None); h_out: where h' goes (default: h itself).  Returns (h', x)."""
    import torch
    ldh = ldo = _rows2d(h, "h")
    shape = h.shape
    R, d = shape
    hcode = _type(h, "h")
    new = []
    if x is None:
        x = torch.empty(R, d, dtype=torch.bfloat16, device=h.device)
        new.append(x)
    elif x.dtype is not torch.bfloat16 or x.shape != shape:
        raise ValueError("x must be a bf16 tensor shaped like h")
    if h_out is None:
        h_out = h
    elif h_out is not h:
        if h_out.dtype is not h.dtype or h_out.shape != shape:
            raise ValueError("h_out must be shaped like h and of its type")
        ldo = _rows2d(h_out, "h_out")
    yp = ycode = ldy = 0
    if y is not None:
        if y.shape != shape:
            raise ValueError("y must be shaped like h")
        yp, ycode, ldy = y.data_ptr(), _type(y, "y"), _rows2d(y, "y")
    wcode = prep = postp = 0
    if pre_weight is not None:
        wcode, prep = _norm_weight(pre_weight, d, "pre_weight"), pre_weight.data_ptr()
    if post_weight is not None:
        code, postp = _norm_weight(post_weight, d, "post_weight"), post_weight.data_ptr()
        if prep and code != wcode:
            raise ValueError("pre_weight and post_weight must have one type")
        wcode = code
    gp = gcode = grow = gcol = 0
    if gate is not None:
        gp, gcode, gs, gt = gate.data_ptr(), _type(gate, "gate"), gate.shape, gate.stride()
        if len(gs) == 1 and gs[0] == d:
            gcol = gt[0]
        elif len(gs) == 2 and gs[0] in (1, R) and gs[1] in (1, d):
            grow = gt[0] if gs[0] > 1 else 0
            gcol = gt[1] if gs[1] > 1 else 0
        else:
            raise ValueError("gate must be [d] or broadcastable [rows][d], got %s" % (tuple(gs),))
    dev = _here(h, x, h_out, y, pre_weight, post_weight, gate)
    rc = _lib.load().msb_block_norm(
        h.data_ptr(), hcode, ldh, yp, ycode, ldy, prep, postp, wcode, 1 if post_norm else 0, gp, gcode, grow, gcol,
        skip_scale, residual_scale, eps, h_out.data_ptr(), ldo, x.data_ptr(), _rows2d(x, "x"), R, d,
        _on(stream, dev, new))
    if rc:
        _check(rc, "block_norm")
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
    if mask is not None:
        _mask(mask, T)
    new = []
    if out is None:
        out = torch.empty_like(x)
        new.append(out)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor shaped like x")
    if workspace is None:
        workspace = DenseWorkspace(dims, T, int8, x.device)
        new.append(workspace.buf)
    dev = _here(x, layer.router_t, out, mask, workspace.buf)
    lib, cd = _lib.load(), dims.c()
    tail = (out.data_ptr(), ctypes.byref(cd), workspace.ptr, workspace.nbytes, _on(stream, dev, new))
    head = (x.data_ptr(), T, _ptr(mask), layer.router_t.data_ptr())
    if int8:
        rc = lib.moe_dense_block_int8(*head, layer.gate_up.data_ptr(), layer.gate_up_scale.data_ptr(),
                                      layer.down.data_ptr(), layer.down_scale.data_ptr(), *tail)
    else:
        rc = lib.moe_dense_block(*head, layer.records.data_ptr(), *tail)
    _check(rc, "moe_dense_block")
    return out
