"""ctypes binding of the int8 linear layer and the experts' operators.

As in _lib: tensors become raw pointers here, sizes, strides, types and
devices are checked before a pointer reaches the library, and the work runs
in the HIP kernels.  All tensors of a call must be on one GPU; the call runs
on that GPU's current stream (or ``stream``) whichever GPU is current.

A decoding step makes many of these calls, each a few microseconds of GPU
work, so the checks are written to cost little: they read each tensor's shape
and strides once, and name it only when they refuse it.
"""
from __future__ import annotations

from ._lib import QigError, _check, _empty as _empty_on, load

torch = None
_lib = None
_TYPES = {}
_SCORES = {"softmax": 0, "sigmoid": 1}


def _start():
    """torch and the library, on the first call (importing the package needs
    neither)."""
    global torch, _lib, _empty, _current, _device, _f32, _i8, _u8, _ws_bytes
    import torch as t
    _lib = load()
    _TYPES.update({t.float32: 0, t.bfloat16: 1, t.float16: 2})
    _empty, _f32, _i8, _u8 = t.empty, t.float32, t.int8, t.uint8
    _ws_bytes = _lib.mmq_workspace_bytes()
    _device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    # the current stream's handle without the Stream object (1 us a call)
    _current = getattr(t._C, "_cuda_getCurrentRawStream", None) or (lambda dev: t.cuda.current_stream(dev).cuda_stream)
    torch = t


def _new(shape, dtype, device, stream):
    """A new tensor for a call on ``stream`` (None: the current one)."""
    if stream is None:
        return _empty(shape, dtype=dtype, device=device)
    return _empty_on(shape, dtype, device, stream)


def _type(t, name):
    code = _TYPES.get(t)
    if code is None:
        raise QigError(f"{name} must be float32, bfloat16 or float16, not {t}")
    return code


def _is(t, dtype, name):
    if t.dtype is not dtype:
        raise QigError(f"{name} must be {dtype}, not {t.dtype}")


def _matrix(t, name):
    """(rows, columns, row stride) of a 2-D tensor with unit column stride."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1 and shape[0] > 0):
        raise QigError(f"{name} must be 2-D with unit column stride")
    rows, cols = shape
    ld = stride[0]
    # a single row may carry any stride: the library takes the width
    return rows, cols, ld if rows > 1 or ld > cols else cols


def _sized(t, name, rows, cols):
    """The row stride of a matrix that must be [rows][cols]."""
    r, c, ld = _matrix(t, name)
    if r != rows or c != cols:
        raise QigError(f"{name} must be [{rows}][{cols}], not {list(t.shape)}")
    return ld


def _vector(t, n, name):
    if t.dtype is _f32 and t.numel() == n and t.is_contiguous():
        return
    _is(t, torch.float32, name)
    if t.numel() != n or not t.is_contiguous():
        raise QigError(f"{name} must be contiguous with {n} elements, not {list(t.shape)}")


def _rows16(t, rows, cols, ld, name):
    """A product reads whole 16-byte units of each int8 row: the last row's
    must lie inside the storage."""
    if rows > 0 and t.storage_offset() + (rows - 1) * ld + (cols + 15) // 16 * 16 > t.untyped_storage().nbytes():
        raise QigError(f"{name}'s storage ends inside the last 16-byte unit of its last row: "
                       f"keep rows of a multiple of 16 bytes")


def _int8_rows(t, name):
    if t.dtype is not _i8:
        _is(t, _i8, name)
    rows, cols, ld = _matrix(t, name)
    if rows <= 1:
        ld = (cols + 15) // 16 * 16
    if cols % 16:
        _rows16(t, rows, cols, ld, name)
    return rows, cols, ld


def _refuse_devices(names, tensors):
    dev = None
    for name, t in zip(names, tensors):
        if t is None:
            continue
        if not t.is_cuda:
            raise QigError(f"{name} must be a GPU tensor")
        if dev is not None and t.device != dev:
            raise QigError(f"{name} is on {t.device}, other tensors of the call on {dev}")
        dev = t.device


def _call(fn, what, names, tensors, stream, args):
    """Check that the tensors (the first of them not None) are on one GPU and
    call fn there."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev or dev < 0:
            _refuse_devices(names, tensors)
    if stream is None:
        handle = _current(dev)
    else:
        on = getattr(stream, "device", None)   # a bare handle does not say
        if on is not None and on.index != dev:
            raise QigError(f"stream is on {on}, the tensors on cuda:{dev}")
        handle = stream.cuda_stream
    if _device() == dev:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc:
        _check(rc, what)


def quantize_i8(x, q=None, s=None, stream=None):
    """x[nt][id] (fp32, bf16 or fp16) -> (q, s): int8 rows and one fp32 scale
    a row.  The q made here has rows of a multiple of 16 bytes (a view of
    width id), as the products need; a given q must too if they are to read
    it.  Use it for activations, and once for the rows of a weight matrix."""
    if torch is None:
        _start()
    xt = _type(x.dtype, "x")
    nt, id_, ldx = _matrix(x, "x")
    if q is None:
        ldq = (id_ + 15) // 16 * 16
        q = _new((nt, ldq), _i8, x.device, stream)
        if ldq != id_:
            q = q[:, :id_]
    else:
        _is(q, torch.int8, "q")
        ldq = _sized(q, "q", nt, id_)
    if s is None:
        s = _new((nt,), _f32, x.device, stream)
    else:
        _vector(s, nt, "s")
    _call(_lib.quantize_i8, "quantize_i8", ("x", "q", "s"), (x, q, s), stream,
          (x.data_ptr(), xt, nt, id_, ldx, q.data_ptr(), ldq, s.data_ptr()))
    return q, s


def _output(y, dtype, nt, od, device, stream):
    """(y, its type's code, row stride)."""
    if y is None:
        dtype = torch.float32 if dtype is None else dtype
        code = _type(dtype, "y")
        return _new((nt, od), dtype, device, stream), code, od
    if dtype is not None and y.dtype != dtype:
        raise QigError(f"y is {y.dtype}, dtype asks for {dtype}")
    code = _type(y.dtype, "y")
    return y, code, _sized(y, "y", nt, od)


def _out_rows(rows, glu):
    if not glu:
        return rows
    if rows % 2:
        raise QigError(f"glu needs an even number of weight rows (gate rows, then up rows), not {rows}")
    return rows // 2


def mm_i8(W, sw, q, sq, bias=None, glu=False, y=None, dtype=None, ws=None, stream=None):
    """y[nt][od] = (q . W^T) * sq * sw + bias from int8 rows q[nt][id] with
    scales sq[nt] and int8 weights W[od][id] with scales sw[od] (quantize_i8
    makes both).  glu: W holds the gate's od rows and then the up's, and y =
    silu(gate) * up.  y is fp32, or of ``dtype`` or the given y's type (bf16,
    fp16).  ws: None, or a workspace (qig.workspace()), which lets a product
    with few output tiles use the whole GPU; y is the same either way."""
    if torch is None:
        _start()
    rows, id_, ldw = _int8_rows(W, "W")
    nt, idq, ldq = _int8_rows(q, "q")
    if idq != id_:
        raise QigError(f"q has {idq} columns, W has {id_}")
    od = _out_rows(rows, glu)
    _vector(sw, rows, "sw")
    _vector(sq, nt, "sq")
    if bias is not None:
        _vector(bias, rows, "bias")
    y, yt, ldy = _output(y, dtype, nt, od, q.device, stream)
    if ws is not None and (ws.numel() * (1 if ws.dtype is _u8 else ws.element_size()) < _ws_bytes
                           or not ws.is_contiguous()):
        raise QigError(f"ws holds {ws.numel() * ws.element_size()} bytes, the call needs {_ws_bytes}, contiguous")
    _call(_lib.mm_i8, "mm_i8", ("W", "sw", "q", "sq", "bias", "y", "ws"), (W, sw, q, sq, bias, y, ws), stream,
          (W.data_ptr(), ldw, sw.data_ptr(), od, id_, q.data_ptr(), ldq, sq.data_ptr(), nt,
           None if bias is None else bias.data_ptr(), 1 if glu else 0, y.data_ptr(), yt, ldy,
           None if ws is None else ws.data_ptr()))
    return y


def route_experts(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renorm=True,
                  scale=1.0, ids=None, w=None, stream=None):
    """logits[nt][ne] -> (ids, w): each token's k experts (int32 [nt][k],
    best first, -1 for a slot that no expert can fill) and their weights
    (fp32 [nt][k]).  score: "softmax" or "sigmoid"; bias [ne] is added to the
    scores for the choice alone; groups > 1 keeps the topk_groups best of that
    many equal runs of experts, a run's score being the sum of its group_top
    largest; renorm divides the weights by their sum; scale multiplies them."""
    if torch is None:
        _start()
    lt = _type(logits.dtype, "logits")
    nt, ne, ldl = _matrix(logits, "logits")
    if score not in _SCORES:
        raise QigError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    if bias is not None:
        _vector(bias, ne, "bias")
    if ids is None:
        ids = _new((nt, max(k, 0)), torch.int32, logits.device, stream)
    else:
        _is(ids, torch.int32, "ids")
        if ids.numel() != nt * k or not ids.is_contiguous():
            raise QigError(f"ids must be contiguous [{nt}][{k}], not {list(ids.shape)}")
    if w is None:
        w = _new((nt, max(k, 0)), _f32, logits.device, stream)
    else:
        _vector(w, nt * k, "w")
    _call(_lib.route_experts, "route_experts", ("logits", "bias", "ids", "w"), (logits, bias, ids, w), stream,
          (logits.data_ptr(), lt, nt, ne, ldl, None if bias is None else bias.data_ptr(), _SCORES[score], groups,
           topk_groups, group_top, k, 1 if renorm else 0, scale, ids.data_ptr(), w.data_ptr()))
    return ids, w


def expert_plan_bytes(nrows: int, ne: int) -> int:
    return int(load().expert_plan_bytes(nrows, ne))


def plan_experts(ids, ne, out=None, stream=None):
    """ids (int32, [nt][k] or flat) -> the order of its rows by expert, as
    int32 words for mm_i8_experts.  Rows whose id is outside [0, ne) have no
    expert."""
    if torch is None:
        _start()
    _is(ids, torch.int32, "ids")
    if not ids.is_contiguous():
        raise QigError("ids must be contiguous")
    n = ids.numel()
    words = _lib.expert_plan_bytes(n, ne) // 4
    if words == 0:
        raise QigError(f"no plan for {n} rows and {ne} experts")
    if out is None:
        out = _new((words,), torch.int32, ids.device, stream)
    else:
        _is(out, torch.int32, "out")
        if out.numel() < words or not out.is_contiguous():
            raise QigError(f"out must be contiguous with at least {words} words")
    _call(_lib.plan_experts, "plan_experts", ("ids", "out"), (ids, out), stream,
          (ids.data_ptr(), n, ne, out.data_ptr()))
    return out


def mm_i8_experts(W, sw, q, sq, plan, nrows, bias=None, glu=False, y=None, dtype=None, stream=None):
    """y[nrows][od]: row r is mm_i8's result for row r // (nrows // len(q)) of
    q and the weights W[e] of row r's expert e, by the plan of the same rows
    (plan_experts); rows without an expert are zeros.  W[ne][od or 2 od][id],
    sw and bias [ne][od or 2 od]."""
    if torch is None:
        _start()
    _is(W, torch.int8, "W")
    shape, stride = W.shape, W.stride()
    if len(shape) != 3 or (shape[2] > 1 and stride[2] != 1):
        raise QigError("W must be [experts][rows][id] with unit stride in the last dimension")
    ne, rows, id_ = shape
    ldw = stride[1] if rows > 1 else stride[0]
    if ne > 1 and rows > 0 and stride[0] != rows * ldw:
        raise QigError("W's experts must follow each other: stride(0) == shape[1] * stride(1)")
    if ne * rows <= 1:
        ldw = (id_ + 15) // 16 * 16
    if id_ % 16:
        _rows16(W, ne * rows, id_, ldw, "W")
    nx, idq, ldq = _int8_rows(q, "q")
    if idq != id_:
        raise QigError(f"q has {idq} columns, W has {id_}")
    if nrows < 0 or (nrows > 0 and (nx == 0 or nrows % nx)):
        raise QigError(f"{nrows} rows are no multiple of the {nx} rows of q")
    slots = nrows // nx if nrows > 0 else 1
    od = _out_rows(rows, glu)
    _vector(sw, ne * rows, "sw")
    _vector(sq, nx, "sq")
    if bias is not None:
        _vector(bias, ne * rows, "bias")
    _is(plan, torch.int32, "plan")
    nbytes = _lib.expert_plan_bytes(nrows, ne)
    if nbytes == 0 or plan.numel() * 4 < nbytes or not plan.is_contiguous():
        raise QigError(f"plan is not one of {nrows} rows and {ne} experts")
    y, yt, ldy = _output(y, dtype, nrows, od, q.device, stream)
    _call(_lib.mm_i8_experts, "mm_i8_experts",
          ("W", "sw", "q", "sq", "plan", "bias", "y"), (W, sw, q, sq, plan, bias, y), stream,
          (W.data_ptr(), ldw, sw.data_ptr(), ne, od, id_, q.data_ptr(), ldq, sq.data_ptr(), nrows, slots,
           plan.data_ptr(), None if bias is None else bias.data_ptr(), 1 if glu else 0, y.data_ptr(), yt, ldy))
    return y


def combine_experts(h, w, y=None, dtype=None, stream=None):
    """y[nt][od] = sum over s of w[t][s] * h[t * k + s] for h[nt * k][od] and
    w[nt][k] (fp32), summed in fp32 in the order of s.  y is of h's type, or of
    ``dtype`` or the given y's type."""
    if torch is None:
        _start()
    ht = _type(h.dtype, "h")
    _is(w, torch.float32, "w")
    if w.dim() != 2 or not w.is_contiguous():
        raise QigError("w must be contiguous [nt][k]")
    nt, k = w.shape
    n, od, ldh = _matrix(h, "h")
    if n != nt * k:
        raise QigError(f"h must be [{nt * k}][any], not {list(h.shape)}")
    y, yt, ldy = _output(y, h.dtype if y is None and dtype is None else dtype, nt, od, h.device, stream)
    _call(_lib.combine_experts, "combine_experts", ("h", "w", "y"), (h, w, y), stream,
          (h.data_ptr(), ht, ldh, w.data_ptr(), nt, k, od, y.data_ptr(), yt, ldy))
    return y
