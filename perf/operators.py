"""Cases, inputs and plain forms of the int8 operators: a linear layer in int8
(activations quantized per token, weights per channel), the routing of tokens
to experts, the experts' products, and one whole experts' layer.

``run`` computes a case in elementary torch operations, or, where ``own`` is
true, through the package's entry points.  ``exact`` computes it in 64 bits
from the definitions:

* quantization of a row: s = max|x| / 127 rounded to fp32, q = the integer
  nearest x / s (ties away from zero), 0 where s = 0;
* product: y = sx * sw * sum(q * w) + bias; gated: a * sigmoid(a) * b with a
  from the first half of the weight rows and b from the second;
* routing: scores s (softmax or sigmoid), choice by s + bias among the experts
  of the best groups, ties to the lowest index, weights from s alone.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def _linear(name, nt, od, id_, x, y, glu=False, bias=False):
    return {"name": name, "op": "linear", "nt": nt, "od": od, "id": id_, "x": x, "y": y, "glu": glu, "bias": bias}


def _route(name, nt, e, k, x, score, groups=1, keep=1, top=1, bias=False, renorm=True):
    return {"name": name, "op": "route", "nt": nt, "e": e, "k": k, "x": x, "score": score, "groups": groups,
            "keep": keep, "top": top, "bias": bias, "renorm": renorm}


def _experts(name, op, nt, e, k, od, id_, x, y):
    return {"name": name, "op": op, "nt": nt, "e": e, "k": k, "od": od, "id": id_, "x": x, "y": y}


def listed():
    return [
        # one new token through a 3584 x 3584 projection: launches and the weights' bytes
        _linear("linear_token", 1, 3584, 3584, "bf16", "bf16"),
        # a batch of decoding requests, sizes that no tile divides, with a bias
        _linear("linear_batch_odd", 37, 1000, 3601, "f16", "f16", bias=True),
        # the headline projection's shape, fp32 in and out as the k-quant products
        _linear("linear_proj", 512, 3584, 3584, "f32", "f32"),
        # a prefill's gate and up projections with the gate applied
        _linear("linear_ffn_gated", 2630, 18944, 3584, "bf16", "bf16", glu=True),
        # a prefill's down projection: the longest sums
        _linear("linear_down", 2630, 3584, 18944, "bf16", "f32"),
        # a prefill's routing, plain top-k of a softmax
        _route("route_softmax", 2630, 64, 6, "f32", "softmax"),
        # many tokens, sigmoid scores with a balance bias and groups
        _route("route_grouped", 16384, 256, 8, "f32", "sigmoid", 8, 4, 2, True),
        # four decoding tokens: nearly every row meets another expert's weights
        _experts("experts_up_token", "up", 4, 64, 6, 2368, 3584, "bf16", "bf16"),
        # a prefill's gate and up products of all experts, an eighth of the dense layer's width each
        _experts("experts_up", "up", 2630, 64, 6, 2368, 3584, "bf16", "bf16"),
        # and their down products, summed with the routing weights
        _experts("experts_down", "down", 2630, 64, 6, 3584, 2368, "bf16", "bf16"),
        # a whole experts' layer: a few decoding requests, and a prompt
        _experts("layer_batch", "layer", 16, 64, 6, 2368, 3584, "bf16", "bf16"),
        _experts("layer_prompt", "layer", 512, 64, 6, 2368, 3584, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "route", "up", "down", "layer"])
    x, y = rng.choice(["f32", "bf16", "f16"]), rng.choice(["f32", "bf16", "f16"])
    if op == "linear":
        nt, od, id_ = _log(rng, 1, 2630), _log(rng, 64, 18944), _log(rng, 64, 18944)
        while nt * od * id_ > 2630 * 3584 * 18944:
            od, id_ = max(64, od // 2), max(64, id_ - id_ // 3)
        c = _linear("", nt, od, id_, x, y, rng.random() < 0.3, rng.random() < 0.3)
    elif op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        e = groups * rng.randint(max(2, 16 // groups), 256 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(12, keep * (e // groups)))
        c = _route("", _log(rng, 1, 16384), e, k, x, rng.choice(["softmax", "sigmoid"]), groups, keep,
                   rng.choice([1, 2]), rng.random() < 0.5, rng.random() < 0.7)
    else:
        e = _log(rng, 4, 64)
        nt, k = _log(rng, 1, 2630 if op != "layer" else 512), rng.randint(1, min(6, e))
        od, id_ = _log(rng, 128, 2368), _log(rng, 128, 3584)
        if op == "down":
            od, id_ = id_, od
        c = _experts("", op, nt, e, k, od, id_, x, y)
    del c["name"]
    return c


# --- inputs ---------------------------------------------------------------------------------------------------------

def _weights(g, shape):
    """int8 weights and their scales per output channel, as a quantization of
    Gaussian weights leaves them (outputs of order one)."""
    w = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    q = w.mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    s = torch.rand(shape[:-1], generator=g, device="cuda").add_(0.5) / (36.0 * math.sqrt(shape[-1]))
    return q, s


def _aligned(q):
    """The weights with rows of a multiple of 16 bytes, as a program keeps
    them: a view of the true width."""
    n = q.shape[-1]
    if n % 16 == 0:
        return q
    p = torch.zeros(q.shape[:-1] + ((n + 15) // 16 * 16,), dtype=q.dtype, device=q.device)
    p[..., :n] = q
    return p[..., :n]


def _activations(g, nt, n, kind):
    """Rows of different size with a few large channels."""
    x = torch.randn((nt, n), generator=g, device="cuda")
    x = x * (torch.rand((nt, 1), generator=g, device="cuda") * 2 + 0.5)
    x = x * (1 + 8 * (torch.rand((1, n), generator=g, device="cuda") > 0.995))
    return x.to(TYPES[kind])


def _logits(g, nt, e, kind):
    popular = torch.randn((1, e), generator=g, device="cuda") * 0.5
    return (torch.randn((nt, e), generator=g, device="cuda") * 1.5 + popular).to(TYPES[kind])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "linear":
        rows = case["od"] * (2 if case["glu"] else 1)
        s["x"] = _activations(g, case["nt"], case["id"], case["x"])
        w, s["sw"] = _weights(g, (rows, case["id"]))
        s["w"] = _aligned(w)
        s["bias"] = torch.randn(rows, generator=g, device="cuda") * 0.3 if case["bias"] else None
    elif case["op"] == "route":
        s["logits"] = _logits(g, case["nt"], case["e"], case["x"])
        s["bias"] = torch.randn(case["e"], generator=g, device="cuda") * 0.1 if case["bias"] else None
    else:
        nt, e, k, od, id_ = (case[n] for n in ("nt", "e", "k", "od", "id"))
        s["logits"] = _logits(g, nt, e, "f32")
        if case["op"] != "layer":
            s["rw"], ids = torch.softmax(s["logits"], 1).topk(k, 1)
            s["ids"] = ids.to(torch.int32)
        s["x"] = _activations(g, nt * (k if case["op"] == "down" else 1), id_, case["x"])
        w, s["sw"] = _weights(g, (e, od * (1 if case["op"] == "down" else 2), id_))
        s["w"] = _aligned(w)
        if case["op"] == "layer":
            w, s["sw2"] = _weights(g, (e, id_, od))
            s["w2"] = _aligned(w)
    return s


# --- plain forms ----------------------------------------------------------------------------------------------------

def _quantize(x):
    """q (as fp32 integers) and s.  The quotient is formed in 64 bits: x / s
    near the border between two integers decides which one it is."""
    x = x.float()
    big = x.abs().amax(1)
    s = big / torch.full_like(big, 127.0)  # a tensor: a division by a number is a product with its rounded inverse
    d = torch.where(s > 0, s, 1.0).double()
    v = x.double() / d[:, None]
    q = torch.sign(v) * torch.floor(v.abs() + 0.5).clamp(max=127.0)
    return q.float(), s


def _gate(y):
    a, b = y.chunk(2, -1)
    return a / (1 + torch.exp(-a)) * b


def _linear_plain(s):
    c = s["case"]
    q, sx = _quantize(s["x"])
    y = (q @ s["w"].float().t()) * sx[:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return (_gate(y) if c["glu"] else y).to(TYPES[c["y"]])


def _route_plain(logits, k, score, groups, keep, top, bias, renorm):
    """Scores in 64 bits: which expert wins is a comparison of near values."""
    v = logits.double()
    p = torch.exp(v - v.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) if score == "softmax" else 1 / (1 + torch.exp(-v))
    c = p if bias is None else p + bias.double()
    if groups > 1:
        best = c.view(c.shape[0], groups, -1).sort(dim=2, descending=True, stable=True)[0]
        order = best[:, :, :top].sum(2).sort(dim=1, descending=True, stable=True)[1]
        lost = torch.ones((c.shape[0], groups), dtype=torch.bool, device=c.device).scatter_(1, order[:, :keep], False)
        c = c.masked_fill(lost.repeat_interleave(c.shape[1] // groups, 1), -math.inf)
    ids = c.sort(dim=1, descending=True, stable=True)[1][:, :k]
    w = p.gather(1, ids)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w.float()


def _products_plain(q, sx, w, sw, ids):
    """Every row with its expert's weights: the rows of each expert gathered
    into one padded batch, one batched product, and back."""
    e, r = w.shape[0], ids.numel()
    flat = ids.reshape(-1).long()
    order = flat.sort(stable=True)[1]
    to = flat[order]
    counts = torch.bincount(flat, minlength=e)
    at = torch.arange(r, device=flat.device) - (counts.cumsum(0) - counts)[to]
    src = order // (r // q.shape[0])
    batch = torch.zeros((e, int(counts.max()), q.shape[1]), device=q.device)
    batch[to, at] = q[src]
    y = torch.bmm(w.float(), batch.transpose(1, 2).contiguous())
    out = torch.empty((r, w.shape[1]), device=q.device)
    out[order] = y.transpose(1, 2)[to, at] * sx[src][:, None] * sw[to]
    return out


def _up_plain(x, w, sw, ids):
    q, sx = _quantize(x)
    return _gate(_products_plain(q, sx, w, sw, ids))


def _down_plain(h, w, sw, ids, rw):
    q, sx = _quantize(h)
    y = _products_plain(q, sx, w, sw, ids)
    return (y.view(rw.shape[0], rw.shape[1], -1) * rw[:, :, None]).sum(1)


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        return _linear_plain(s)
    if c["op"] == "route":
        return _route_plain(s["logits"], c["k"], c["score"], c["groups"], c["keep"], c["top"], s["bias"], c["renorm"])
    out = TYPES[c["y"]]
    if c["op"] == "up":
        return _up_plain(s["x"], s["w"], s["sw"], s["ids"]).to(out)
    if c["op"] == "down":
        return _down_plain(s["x"], s["w"], s["sw"], s["ids"], s["rw"]).to(out)
    ids, rw = _route_plain(s["logits"], c["k"], "softmax", 1, 1, 1, None, True)
    h = _up_plain(s["x"], s["w"], s["sw"], ids)
    return [ids, _down_plain(h, s["w2"], s["sw2"], ids, rw).to(out)]


# --- the package's calls --------------------------------------------------------------------------------------------

def _own(s):
    import quant_integer_gemm_amd as qig
    c = s["case"]
    if c["op"] == "linear":
        q, sx = qig.quantize_i8(s["x"])
        return qig.mm_i8(s["w"], s["sw"], q, sx, bias=s["bias"], glu=c["glu"], dtype=TYPES[c["y"]],
                         ws=qig.workspace(q.device))
    if c["op"] == "route":
        return qig.route_experts(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                 topk_groups=c["keep"], group_top=c["top"], renorm=c["renorm"])
    out, rows = TYPES[c["y"]], c["nt"] * c["k"]
    if c["op"] == "layer":
        ids, rw = qig.route_experts(s["logits"], c["k"])
    else:
        ids, rw = s["ids"], s.get("rw")
    plan = qig.plan_experts(ids, c["e"])
    q, sx = qig.quantize_i8(s["x"])
    if c["op"] == "up":
        return qig.mm_i8_experts(s["w"], s["sw"], q, sx, plan, rows, glu=True, dtype=out)
    if c["op"] == "down":
        # the rows stay in fp32 until they are summed: one rounding at the end
        h = qig.mm_i8_experts(s["w"], s["sw"], q, sx, plan, rows)
        return qig.combine_experts(h, rw, dtype=out)
    h = qig.mm_i8_experts(s["w"], s["sw"], q, sx, plan, rows, glu=True)
    q, sx = qig.quantize_i8(h)
    h = qig.mm_i8_experts(s["w2"], s["sw2"], q, sx, plan, rows)
    return [ids, qig.combine_experts(h, rw, dtype=out)]


def run(state):
    return _own(state) if own else _plain(state)


# --- the work of a pass ---------------------------------------------------------------------------------------------

def _touched(e, rows, k):
    """Experts that some row meets, when tokens choose evenly."""
    return e * (1 - (1 - k / e) ** max(1, rows // k)) if k < e else e


def work(case):
    c, op = case, case["op"]
    if op == "linear":
        rows = c["od"] * (2 if c["glu"] else 1)
        return {"bytes": c["nt"] * c["id"] * BYTES[c["x"]] + rows * (c["id"] + 4) + c["nt"] * c["od"] * BYTES[c["y"]],
                "flops": 2 * c["nt"] * rows * c["id"]}
    if op == "route":
        return {"bytes": c["nt"] * (c["e"] * BYTES[c["x"]] + 8 * c["k"]), "flops": 8 * c["nt"] * c["e"]}
    nt, k, od, id_, r = c["nt"], c["k"], c["od"], c["id"], c["nt"] * c["k"]
    e = _touched(c["e"], r, k)
    if op == "up":
        return {"bytes": int(nt * id_ * BYTES[c["x"]] + e * 2 * od * (id_ + 4) + r * (od * BYTES[c["y"]] + 4)),
                "flops": 4 * r * od * id_}
    if op == "down":
        return {"bytes": int(r * (id_ * BYTES[c["x"]] + 8) + e * od * (id_ + 4) + nt * od * BYTES[c["y"]]),
                "flops": 2 * r * od * id_}
    return {"bytes": int(nt * (c["e"] * 4 + id_ * (BYTES[c["x"]] + BYTES[c["y"]])) + e * 3 * od * id_ + r * 4),
            "flops": 6 * r * od * id_}


# --- 64 bits, from the definitions ----------------------------------------------------------------------------------

def _exact_rows(x):
    x = x.to(torch.float64)
    big = x.abs().max(dim=1, keepdim=True).values
    s = (big / 127).to(torch.float32).to(torch.float64)
    q = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    q = torch.copysign((q.abs() * 2 + 1).div(2).floor(), q).clamp(-127, 127)
    return q, s


def _exact_silu(a):
    return a * torch.special.expit(a)


def _exact_experts(x, w, sw, ids, gated):
    q, s = _exact_rows(x)
    r = ids.numel()
    rep = r // x.shape[0]
    e_of = ids.reshape(-1).tolist()
    rows = [[] for _ in range(w.shape[0])]
    for i, e in enumerate(e_of):
        rows[e].append(i)
    od = w.shape[1] // 2 if gated else w.shape[1]
    out = torch.zeros((r, od), dtype=torch.float64, device=x.device)
    for e, mine in enumerate(rows):
        if not mine:
            continue
        mine = torch.tensor(mine, device=x.device)
        src = torch.div(mine, rep, rounding_mode="floor")
        y = torch.matmul(q[src], w[e].to(torch.float64).T.contiguous()) * sw[e].to(torch.float64) * s[src]
        out[mine] = _exact_silu(y[:, :od]) * y[:, od:] if gated else y
    return out


def _exact_route(c, logits, bias):
    l = logits.to(torch.float64).cpu()
    p = torch.softmax(l, dim=-1) if c["score"] == "softmax" else torch.special.expit(l)
    choice = p.clone() if bias is None else p + bias.to(torch.float64).cpu()
    size = choice.shape[1] // c["groups"]
    if c["groups"] > 1:
        per = torch.stack([part.topk(min(c["top"], size), dim=1).values.sum(1) for part in choice.split(size, 1)], 1)
        for _ in range(c["groups"] - c["keep"]):
            # the worst group goes, the last one of equals
            worst = per.shape[1] - 1 - per.flip(1).argmin(1)
            per[torch.arange(len(per)), worst] = math.inf
        choice[torch.isinf(per).repeat_interleave(size, 1)] = -math.inf
    ids = []
    for _ in range(c["k"]):
        top = choice.max(1, keepdim=True).values
        first = (choice == top).to(torch.uint8).argmax(1)
        ids.append(first)
        choice[torch.arange(len(first)), first] = -math.inf
    ids = torch.stack(ids, 1)
    w = torch.take_along_dim(p, ids, 1)
    return ids, w / w.sum(1, keepdim=True) if c["renorm"] else w


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        q, sx = _exact_rows(s["x"])
        y = torch.matmul(q, s["w"].to(torch.float64).T.contiguous()) * sx * s["sw"].to(torch.float64)
        if s["bias"] is not None:
            y += s["bias"].to(torch.float64)
        return _exact_silu(y[:, :c["od"]]) * y[:, c["od"]:] if c["glu"] else y
    if c["op"] == "route":
        return [None, _exact_route(c, s["logits"], s["bias"])[1]]
    if c["op"] == "up":
        return _exact_experts(s["x"], s["w"], s["sw"], s["ids"], True)
    if c["op"] == "layer":
        plain = {"score": "softmax", "groups": 1, "keep": 1, "top": 1, "renorm": True, "k": c["k"]}
        ids, rw = (t.to(s["x"].device) for t in _exact_route(plain, s["logits"], None))
        h = _exact_experts(s["x"], s["w"], s["sw"], ids, True)
        y = _exact_experts(h, s["w2"], s["sw2"], ids, False)
    else:
        rw = s["rw"].to(torch.float64)
        y = _exact_experts(s["x"], s["w"], s["sw"], s["ids"], False)
    y = (y.view(rw.shape[0], rw.shape[1], -1) * rw[..., None]).sum(1)
    return [None, y] if c["op"] == "layer" else y
