"""ctypes binding of the int8 linear layer and the experts' operators.

As in _lib: tensors become raw pointers here, sizes, strides, types and
devices are checked before a pointer reaches the library, and the work runs
in the HIP kernels.  All tensors of a call must be on one GPU; the call runs
on that GPU's current stream (or ``stream``) whichever GPU is current.
"""
from __future__ import annotations

import ctypes

from ._lib import QigError, _check, _dev_ptr, load

_SCORES = {"softmax": 0, "sigmoid": 1}


def _type(t, name):
    import torch
    code = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}.get(t)
    if code is None:
        raise QigError(f"{name} must be float32, bfloat16 or float16, not {t}")
    return code


def _is(t, dtype, name):
    if t.dtype != dtype:
        raise QigError(f"{name} must be {dtype}, not {t.dtype}")


def _matrix(t, name, rows=None, cols=None):
    """(rows, columns, row stride) of a 2-D tensor with unit column stride."""
    if t.dim() != 2 or (t.numel() > 0 and t.shape[1] > 1 and t.stride(1) != 1):
        raise QigError(f"{name} must be 2-D with unit column stride")
    if (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise QigError(f"{name} must be [{'any' if rows is None else rows}][{'any' if cols is None else cols}], "
                       f"not {list(t.shape)}")
    # a single row may carry any stride: the library takes the width
    return t.shape[0], t.shape[1], t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _vector(t, n, name):
    import torch
    if t is None:
        return
    _is(t, torch.float32, name)
    if t.numel() != n or not t.is_contiguous():
        raise QigError(f"{name} must be contiguous with {n} elements, not {list(t.shape)}")


def _rows16(t, cols, ld, name):
    """A product reads whole 16-byte units of each int8 row: the last row's
    must lie inside the storage."""
    rows = t.numel() // max(cols, 1)
    if rows > 0 and t.storage_offset() + (rows - 1) * ld + (cols + 15) // 16 * 16 > t.untyped_storage().nbytes():
        raise QigError(f"{name}'s storage ends inside the last 16-byte unit of its last row: "
                       f"keep rows of a multiple of 16 bytes")


def _int8_rows(t, name):
    import torch
    _is(t, torch.int8, name)
    rows, cols, ld = _matrix(t, name)
    if rows <= 1:
        ld = (cols + 15) // 16 * 16
    _rows16(t, cols, ld, name)
    return rows, cols, ld


def _run(fn, what, tensors, stream, *args):
    """Check that the tensors are on one GPU and call fn there."""
    import torch
    dev = None
    for name, t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise QigError(f"{name} must be a GPU tensor")
        if dev is not None and t.device != dev:
            raise QigError(f"{name} is on {t.device}, other tensors of the call on {dev}")
        dev = t.device
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise QigError(f"stream is on {stream.device}, the tensors on {dev}")
    handle = ctypes.c_void_p(stream.cuda_stream)
    if torch.cuda.current_device() == dev.index:
        _check(fn(*args, handle), what)
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, handle), what)


def quantize_i8(x, q=None, s=None, stream=None):
    """x[nt][id] (fp32, bf16 or fp16) -> (q, s): int8 rows and one fp32 scale
    a row.  The q made here has rows of a multiple of 16 bytes (a view of
    width id), as the products need; a given q must too if they are to read
    it.  Use it for activations, and once for the rows of a weight matrix."""
    import torch
    xt = _type(x.dtype, "x")
    nt, id_, ldx = _matrix(x, "x")
    if q is None:
        q = torch.empty((nt, (id_ + 15) // 16 * 16), dtype=torch.int8, device=x.device)[:, :id_]
    _is(q, torch.int8, "q")
    ldq = _matrix(q, "q", nt, id_)[2]
    if s is None:
        s = torch.empty(nt, dtype=torch.float32, device=x.device)
    _vector(s, nt, "s")
    _run(load().quantize_i8, "quantize_i8", (("x", x), ("q", q), ("s", s)), stream,
         _dev_ptr(x, "x"), xt, nt, id_, ldx, _dev_ptr(q, "q"), ldq, _dev_ptr(s, "s"))
    return q, s


def _output(y, dtype, nt, od, device):
    import torch
    if y is None:
        y = torch.empty((nt, od), dtype=torch.float32 if dtype is None else dtype, device=device)
    elif dtype is not None and y.dtype != dtype:
        raise QigError(f"y is {y.dtype}, dtype asks for {dtype}")
    yt = _type(y.dtype, "y")
    return y, yt, _matrix(y, "y", nt, od)[2]


def _out_rows(rows, glu):
    if glu and rows % 2:
        raise QigError(f"glu needs an even number of weight rows (gate rows, then up rows), not {rows}")
    return rows // 2 if glu else rows


def mm_i8(W, sw, q, sq, bias=None, glu=False, y=None, dtype=None, ws=None, stream=None):
    """y[nt][od] = (q . W^T) * sq * sw + bias from int8 rows q[nt][id] with
    scales sq[nt] and int8 weights W[od][id] with scales sw[od] (quantize_i8
    makes both).  glu: W holds the gate's od rows and then the up's, and y =
    silu(gate) * up.  y is fp32, or of ``dtype`` or the given y's type (bf16,
    fp16).  ws: None, or a workspace (qig.workspace()), which lets a product
    with few output tiles use the whole GPU; y is the same either way."""
    from ._lib import _need
    rows, id_, ldw = _int8_rows(W, "W")
    nt, idq, ldq = _int8_rows(q, "q")
    if idq != id_:
        raise QigError(f"q has {idq} columns, W has {id_}")
    od = _out_rows(rows, glu)
    _vector(sw, rows, "sw")
    _vector(bias, rows, "bias")
    _vector(sq, nt, "sq")
    y, yt, ldy = _output(y, dtype, nt, od, q.device)
    if ws is not None:
        _need(ws, int(load().mmq_workspace_bytes()), "ws")
    _run(load().mm_i8, "mm_i8",
         (("W", W), ("sw", sw), ("q", q), ("sq", sq), ("bias", bias), ("y", y), ("ws", ws)), stream,
         _dev_ptr(W, "W"), ldw, _dev_ptr(sw, "sw"), od, id_, _dev_ptr(q, "q"), ldq, _dev_ptr(sq, "sq"), nt,
         _dev_ptr(bias, "bias"), int(bool(glu)), _dev_ptr(y, "y"), yt, ldy, _dev_ptr(ws, "ws"))
    return y


def route_experts(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renorm=True,
                  scale=1.0, ids=None, w=None, stream=None):
    """logits[nt][ne] -> (ids, w): each token's k experts (int32 [nt][k],
    best first, -1 for a slot that no expert can fill) and their weights
    (fp32 [nt][k]).  score: "softmax" or "sigmoid"; bias [ne] is added to the
    scores for the choice alone; groups > 1 keeps the topk_groups best of that
    many equal runs of experts, a run's score being the sum of its group_top
    largest; renorm divides the weights by their sum; scale multiplies them."""
    import torch
    lt = _type(logits.dtype, "logits")
    nt, ne, ldl = _matrix(logits, "logits")
    if score not in _SCORES:
        raise QigError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    _vector(bias, ne, "bias")
    if ids is None:
        ids = torch.empty((nt, max(k, 0)), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((nt, max(k, 0)), dtype=torch.float32, device=logits.device)
    _is(ids, torch.int32, "ids")
    _vector(w, nt * k, "w")
    if ids.numel() != nt * k or not ids.is_contiguous():
        raise QigError(f"ids must be contiguous [{nt}][{k}], not {list(ids.shape)}")
    _run(load().route_experts, "route_experts", (("logits", logits), ("bias", bias), ("ids", ids), ("w", w)), stream,
         _dev_ptr(logits, "logits"), lt, nt, ne, ldl, _dev_ptr(bias, "bias"), _SCORES[score], groups, topk_groups,
         group_top, k, int(bool(renorm)), float(scale), _dev_ptr(ids, "ids"), _dev_ptr(w, "w"))
    return ids, w


def expert_plan_bytes(nrows: int, ne: int) -> int:
    return int(load().expert_plan_bytes(nrows, ne))


def plan_experts(ids, ne, out=None, stream=None):
    """ids (int32, [nt][k] or flat) -> the order of its rows by expert, as
    int32 words for mm_i8_experts.  Rows whose id is outside [0, ne) have no
    expert."""
    import torch
    _is(ids, torch.int32, "ids")
    if not ids.is_contiguous():
        raise QigError("ids must be contiguous")
    n = ids.numel()
    nbytes = expert_plan_bytes(n, ne)
    if nbytes == 0:
        raise QigError(f"no plan for {n} rows and {ne} experts")
    if out is None:
        out = torch.empty(nbytes // 4, dtype=torch.int32, device=ids.device)
    _is(out, torch.int32, "out")
    if out.numel() * 4 < nbytes or not out.is_contiguous():
        raise QigError(f"out must be contiguous with at least {nbytes // 4} words")
    _run(load().plan_experts, "plan_experts", (("ids", ids), ("out", out)), stream,
         _dev_ptr(ids, "ids"), n, ne, _dev_ptr(out, "plan"))
    return out


def mm_i8_experts(W, sw, q, sq, plan, nrows, bias=None, glu=False, y=None, dtype=None, stream=None):
    """y[nrows][od]: row r is mm_i8's result for row r // (nrows // len(q)) of
    q and the weights W[e] of row r's expert e, by the plan of the same rows
    (plan_experts); rows without an expert are zeros.  W[ne][od or 2 od][id],
    sw and bias [ne][od or 2 od]."""
    import torch
    _is(W, torch.int8, "W")
    if W.dim() != 3 or (W.shape[2] > 1 and W.stride(2) != 1):
        raise QigError("W must be [experts][rows][id] with unit stride in the last dimension")
    ne, rows, id_ = W.shape
    ldw = W.stride(1) if rows > 1 else W.stride(0)
    if ne > 1 and W.stride(0) != rows * ldw:
        raise QigError("W's experts must follow each other: stride(0) == shape[1] * stride(1)")
    if rows == 1 and ne == 1:
        ldw = (id_ + 15) // 16 * 16
    _rows16(W, id_, ldw, "W")
    nx, idq, ldq = _int8_rows(q, "q")
    if idq != id_:
        raise QigError(f"q has {idq} columns, W has {id_}")
    if nrows < 0 or (nrows > 0 and (nx == 0 or nrows % nx)):
        raise QigError(f"{nrows} rows are no multiple of the {nx} rows of q")
    slots = nrows // nx if nrows > 0 else 1
    od = _out_rows(rows, glu)
    _vector(sw, ne * rows, "sw")
    _vector(bias, ne * rows, "bias")
    _vector(sq, nx, "sq")
    _is(plan, torch.int32, "plan")
    nbytes = expert_plan_bytes(nrows, ne)
    if nbytes == 0 or plan.numel() * 4 < nbytes or not plan.is_contiguous():
        raise QigError(f"plan is not one of {nrows} rows and {ne} experts")
    y, yt, ldy = _output(y, dtype, nrows, od, q.device)
    _run(load().mm_i8_experts, "mm_i8_experts",
         (("W", W), ("sw", sw), ("q", q), ("sq", sq), ("plan", plan), ("bias", bias), ("y", y)), stream,
         _dev_ptr(W, "W"), ldw, _dev_ptr(sw, "sw"), ne, od, id_, _dev_ptr(q, "q"), ldq, _dev_ptr(sq, "sq"), nrows,
         slots, _dev_ptr(plan, "plan"), _dev_ptr(bias, "bias"), int(bool(glu)), _dev_ptr(y, "y"), yt, ldy)
    return y


def combine_experts(h, w, y=None, dtype=None, stream=None):
    """y[nt][od] = sum over s of w[t][s] * h[t * k + s] for h[nt * k][od] and
    w[nt][k] (fp32), summed in fp32 in the order of s.  y is of h's type, or of
    ``dtype`` or the given y's type."""
    import torch
    ht = _type(h.dtype, "h")
    _is(w, torch.float32, "w")
    if w.dim() != 2 or not w.is_contiguous():
        raise QigError("w must be contiguous [nt][k]")
    nt, k = w.shape
    _, od, ldh = _matrix(h, "h", nt * k)
    y, yt, ldy = _output(y, h.dtype if y is None and dtype is None else dtype, nt, od, h.device)
    _run(load().combine_experts, "combine_experts", (("h", h), ("w", w), ("y", y)), stream,
         _dev_ptr(h, "h"), ht, ldh, _dev_ptr(w, "w"), nt, k, od, _dev_ptr(y, "y"), yt, ldy)
    return y
