"""Cases, inputs and plain forms of the attention operators: attention over a
whole prompt, a paged cache of keys and values in 4 bits with the attention
that reads it, and the pages' own operators (taking, freeing, forking, copying,
compacting).

``run`` computes a case in elementary torch operations, or, where ``own`` is
true, through the package's entry points.  ``exact`` computes it in 64 bits
from the definitions:

* attention: y = sum_j p_j v_j, p = softmax_j(scale * q . k_j) over the keys
  that a query sees; query i of n sees the keys before length - n + i + 1 (all
  of them where it is not causal); heads share keys in equal groups;
* 4 bits: 32 values of a row with lowest lo and highest hi become
  m = the largest bf16 <= lo, s = the smallest bf16 >= (hi - m) / 15 and
  c = floor((x - m) / s + 1/2) held to 0 .. 15; they stand for m + s * c;
* pages: a row of the table lists the pages of a sequence, -1 for none, and
  refs counts the rows that hold a page.  Free pages are given out lowest first,
  in the order of rows and then of their entries.

The cache's layout: pages [npages][heads][page / 32 blocks][10 d words], a block
holding 32 tokens of one head.  Token 16 u + 4 h + i (u < 2, h < 4, i < 4):
* keys, words 0 .. 4 d: channel 32 g + 8 e + 2 b + a stands in the 4 bits from
  16 a + 4 b on of word ((w / 4) * 64 + e * 16 + 4 h + i) * 4 + w % 4 with
  w = u * d / 32 + g;
* values, words 4 d .. 8 d: channel 16 (4 n + b) + l in the 4 bits from
  16 (i % 2) + 4 b on of word ((w / 4) * 64 + h * 16 + l) * 4 + w % 4 with
  w = (2 u + i / 2) * d / 64 + n;
* scales, words 8 d .. 9 d for keys and 9 d .. 10 d for values: group g in word
  (h * 8 + u * 4 + i) * d / 32 + g, s in the low and m in the high 16 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def _prompt(name, nseq, longest, prefix, hq, hkv, d, x, causal=True, ragged=0):
    return {"name": name, "op": "prompt", "nseq": nseq, "longest": longest, "prefix": prefix, "hq": hq, "hkv": hkv,
            "d": d, "x": x, "causal": causal, "ragged": ragged}


def _cache(name, op, nseq, new, longest, page, hq, hkv, d, x, ragged=0):
    return {"name": name, "op": op, "nseq": nseq, "new": new, "longest": longest, "page": page, "hq": hq, "hkv": hkv,
            "d": d, "x": x, "ragged": ragged}


def _pages(name, rows, width, npages, words, frees, forks, copies, grow, compact):
    return {"name": name, "op": "pages", "rows": rows, "width": width, "npages": npages, "words": words,
            "frees": frees, "forks": forks, "copies": copies, "grow": grow, "compact": compact}


def listed():
    return [
        # a short question alone: 28 query heads on 4 key heads of 128, the widths of the layer's projections
        _prompt("prompt_short", 1, 33, 0, 28, 4, 128, "bf16"),
        # the whole layer's prompt on the k-quant products' fp32 outputs
        _prompt("prompt_layer_f32", 1, 2630, 0, 28, 4, 128, "f32"),
        # many prompts of different lengths in one batch, the later parts of longer ones among them: keys before the queries'
        _prompt("prompt_packed", 24, 999, 700, 32, 8, 64, "f16", ragged=1),
        # a long document
        _prompt("prompt_long", 1, 8191, 0, 28, 4, 128, "bf16"),
        # the decoding step of 64 requests: one token each into the cache, and its values read back
        _cache("write_tokens", "write", 64, 1, 4096, 64, 28, 4, 128, "bf16", ragged=2),
        # a whole prompt into the cache, from fp32 projections
        _cache("write_prompt", "write", 1, 2630, 2630, 64, 28, 4, 128, "f32"),
        # one request that decodes alone
        _cache("attend_token", "attend", 1, 1, 4099, 64, 28, 4, 128, "bf16"),
        # a full batch of requests of very different lengths
        _cache("attend_batch", "attend", 64, 1, 16384, 64, 28, 4, 128, "bf16", ragged=3),
        # drafted tokens that are checked together: five queries a request, each seeing the ones before it
        _cache("attend_drafts", "attend", 16, 5, 3000, 32, 32, 8, 64, "f16", ragged=4),
        # one step of a small server: a request ends, others fork, all grow, and the pool is packed
        _pages("pages_small", 16, 16, 512, 2560, 2, 2, 2, 1, True),
        # the step of a busy server: beams fork, requests end and grow by drafted tokens, shared pages are copied out
        _pages("pages_busy", 512, 128, 16384, 10240, 64, 64, 128, 5, False),
        # a third of the requests gone, the rest packed to the pool's front
        _pages("pages_compact", 1024, 64, 16384, 10240, 340, 0, 0, 0, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "write", "attend", "attend", "attend", "pages", "pages"])
    x, ragged = rng.choice(["f32", "bf16", "f16"]), rng.randint(1, 1 << 30)
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 7, 8])
    if op == "prompt":
        nseq = _log(rng, 1, 32)
        longest, prefix = _log(rng, 1, 8191), rng.choice([0, 0, 1]) * _log(rng, 1, 2048)
        while nseq * longest * (longest + prefix) * hq > (28 << 26) / (4 if x == "f32" else 1):
            longest, prefix, nseq = max(1, longest * 3 // 4), prefix * 3 // 4, max(1, nseq * 3 // 4)
        c = _prompt("", nseq, longest, prefix, hq, hkv, rng.choice([64, 80, 96, 128, 128]), x, rng.random() < 0.8, ragged)
    elif op == "pages":
        rows, width = _log(rng, 4, 1024), _log(rng, 4, 128)
        words = 4 * _log(rng, 64, 2560)
        npages = max(16, min(32768, rows * width * rng.randint(2, 9) // 8, (671 << 20) // (4 * words)))
        c = _pages("", rows, width, npages, words, rng.randint(0, rows // 3), rng.randint(0, rows // 4),
                   rng.randint(0, min(64, npages // 16)), rng.randint(0, 9), rng.random() < 0.6)
    else:
        nseq = _log(rng, 1, 128)
        new = 1 if rng.random() < 0.5 else _log(rng, 1, 8 if op == "attend" else 2630)
        longest = new + _log(rng, 1, 32768)
        while nseq * longest * hkv > 64 * 16384 * 4 or nseq * new * longest * hq > 64 * 8 * 16384 * 28:
            nseq, longest = max(1, nseq * 3 // 4), max(new, longest * 3 // 4)
            new = min(new, longest)
        c = _cache("", op, nseq, new, longest, rng.choice([32, 64, 128]), hq, hkv, rng.choice([64, 128, 128]), x, ragged)
    del c["name"]
    return c


# --- lengths --------------------------------------------------------------------------------------------------------

def _lens(case, longest, least, salt=0):
    """The sequences' lengths: one of them the longest, the others between that
    and the least by their logarithm."""
    if not case["ragged"]:
        return [longest] * case["nseq"]
    rng = random.Random(case["ragged"] * 4 + salt)
    lens = [_log(rng, max(1, least), max(1, longest)) for _ in range(case["nseq"])]
    lens[rng.randrange(len(lens))] = longest
    return lens


def _prompt_lens(case):
    """Queries and keys of each prompt."""
    n = _lens(case, case["longest"], case["longest"] // 16)
    before = _lens(case, case["prefix"], 1, 1) if case["prefix"] else [0] * case["nseq"]
    return n, [a + b for a, b in zip(n, before)]


def _cache_lens(case):
    """New tokens and all tokens of each sequence."""
    n = [case["new"]] * case["nseq"]
    return n, [max(a, b) for a, b in zip(n, _lens(case, case["longest"], case["longest"] // 16))]


def _starts(lens, device="cuda"):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=device)


# --- inputs ---------------------------------------------------------------------------------------------------------

def _heads(g, nt, h, d, spread, kind="f32"):
    """Rows of heads: Gaussian, with offsets and sizes by channel as
    projections leave them."""
    x = torch.randn((nt, h, d), generator=g, device="cuda")
    x *= torch.rand((1, h, d), generator=g, device="cuda") * spread + 0.5
    x += torch.randn((1, h, d), generator=g, device="cuda") * 0.3
    return x.to(TYPES[kind])


def _filled(case, g, lens):
    """Pages that hold the sequences, in no order, and their tables."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    counts = [(n + page - 1) // page for n in lens]
    npages = sum(counts) + 8
    order = torch.randperm(npages, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), max(counts)), -1, dtype=torch.int32, device="cuda")
    cols = torch.arange(max(counts), device="cuda")
    held = torch.tensor(counts, device="cuda")
    mine = cols < held[:, None]
    tables[mine] = order[:sum(counts)]
    pages = torch.zeros((npages, hkv, page // 32 * 40 * d), dtype=torch.uint8, device="cuda")
    return pages, tables


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "prompt":
        n, nk = _prompt_lens(case)
        s["starts"], s["k_starts"] = _starts(n), _starts(nk)
        s["q"] = _heads(g, sum(n), case["hq"], case["d"], 1.0, case["x"])
        s["k"] = _heads(g, sum(nk), case["hkv"], case["d"], 1.0, case["x"])
        s["v"] = _heads(g, sum(nk), case["hkv"], case["d"], 0.5, case["x"])
    elif case["op"] == "pages":
        s.update(_pool(case, g))
    else:
        n, lens = _cache_lens(case)
        s["pages"], s["tables"] = _filled(case, g, lens)
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["starts"] = _starts(n)
        if case["op"] == "write":
            s["k"] = _heads(g, sum(n), case["hkv"], case["d"], 1.0, case["x"])
            s["v"] = _heads(g, sum(n), case["hkv"], case["d"], 0.5, case["x"])
        else:
            s["q"] = _heads(g, sum(n), case["hq"], case["d"], 1.0, case["x"])
            k = _heads(g, sum(lens), case["hkv"], case["d"], 1.0)
            v = _heads(g, sum(lens), case["hkv"], case["d"], 0.5)
            _write_plain(k, v, s["pages"], s["tables"], s["lengths"], _starts(lens), case["page"])
    return s


def _pool(case, g):
    """A pool in use: nine rows of ten hold sequences of different lengths, some
    begin with pages of the row before, and the pages lie scattered.  All
    integers of the pool stand in one tensor: tables, lengths, refs."""
    rows, width, npages, page = case["rows"], case["width"], case["npages"], 32
    used = max(1, rows * 9 // 10)
    rng = random.Random(int(torch.randint(1 << 30, (1,), generator=g, device="cuda")))
    order = list(range(npages))
    rng.shuffle(order)
    spare = case["copies"] + npages // 8   # the last ones of the shuffled order stay free
    tables = [[-1] * width for _ in range(rows)]
    lengths, refs, at = [0] * rows, [0] * npages, 0
    slots = list(range(rows))
    rng.shuffle(slots)
    live = []
    for r in slots[:used]:
        n = min(_log(rng, 1, width), npages - spare - at)
        if n <= 0:
            break
        shared = tables[live[-1]][:max(0, min(n, lengths[live[-1]] // page) // 2)] if live and rng.random() < 0.2 else []
        tables[r][:n] = shared + order[at:at + n - len(shared)]
        at += n - len(shared)
        lengths[r] = n * page - (rng.randrange(page) if n > len(shared) else 0)
        for p in tables[r][:n]:
            refs[p] += 1
        live.append(r)
    rng.shuffle(live)
    frees = live[:min(case["frees"], len(live) // 2)]
    stay = live[len(frees):]
    room = [r for r in range(rows) if lengths[r] == 0] + frees
    forks = min(case["forks"], len(room))
    parents, children = [rng.choice(stay) for _ in range(forks)], rng.sample(room, forks)
    src = [tables[rng.choice(stay)][0] for _ in range(case["copies"])]
    dst = order[npages - case["copies"]:]   # pages outside of every sequence, held by who asked for the copies
    for p in dst:
        refs[p] = 1
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    flat = [p for row in tables for p in row]
    grown = [case["grow"] if r in set(stay) else 0 for r in range(rows)]
    pages = torch.randint(-(1 << 31), (1 << 31) - 1, (npages, case["words"]), generator=g, device="cuda",
                          dtype=torch.int32)
    return {"pages": pages, "held": dev(flat + lengths + refs), "rows": dev(frees), "parents": dev(parents),
            "children": dev(children), "src": dev(src), "dst": dev(dst), "grown": dev(grown), "page": page}


# --- plain forms: attention -----------------------------------------------------------------------------------------

def _spread(x, starts, longest):
    """Packed rows [nt][h][d] to [nseq][h][longest][d] in 32 bits; rows past a
    sequence's end repeat some other row."""
    at = starts[:-1, None].long() + torch.arange(longest, device=x.device)
    at = at.clamp(max=x.shape[0] - 1)
    return x[at].float().transpose(1, 2).contiguous()


def _attend_plain(q, k, v, nq, nk, scale, causal):
    """q [nseq][hq][lq][d], k and v [nseq][hkv][lk][d] in 32 bits, the true
    lengths on the device.  Rows that see no key give zeros."""
    b, hq, lq, d = q.shape
    hkv, lk = k.shape[1], k.shape[2]
    s = torch.matmul(q.view(b, hkv, -1, d), k.transpose(2, 3).contiguous()).view(b, hkv, hq // hkv, lq, lk)
    s.mul_(scale)
    j, i = torch.arange(lk, device=q.device), torch.arange(lq, device=q.device)
    end = (nk - nq)[:, None] + i + 1 if causal else nk[:, None].expand(b, lq)
    seen = j < torch.minimum(end, nk[:, None])[:, :, None]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(4, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(4, keepdim=True)
    y = torch.matmul(p.view(b, hkv, -1, lk), v).view(b, hkv, hq // hkv, lq, d)
    return (y / torch.where(total > 0, total, 1.0)).view(b, hq, lq, d)


def _packed(y, starts, nt):
    """[nseq][h][lq][d] back to packed rows [nt][h][d]."""
    t = torch.arange(nt, device=y.device)
    seq = torch.searchsorted(starts, t, right=True) - 1
    return y.transpose(1, 2)[seq, t - starts[seq]]


def _prompt_plain(s):
    c = s["case"]
    n, nk = _prompt_lens(c)
    lens = lambda starts: starts[1:].long() - starts[:-1].long()  # noqa: E731
    y = _attend_plain(_spread(s["q"], s["starts"], max(n)), _spread(s["k"], s["k_starts"], max(nk)),
                      _spread(s["v"], s["k_starts"], max(nk)), lens(s["starts"]), lens(s["k_starts"]),
                      1 / math.sqrt(c["d"]), c["causal"])
    return _packed(y, s["starts"], s["q"].shape[0]).to(TYPES[c["x"]])


# --- plain forms: the cache -----------------------------------------------------------------------------------------

def _floor_bf16(x):
    """The largest bf16 that is not above x (32 bits): the low half of the
    pattern goes, and a negative number with something there is one step more."""
    bits = x.view(torch.int32)
    low = bits & 0xffff
    up = ((bits < 0) & (low != 0)).int() << 16
    return (bits - low + up).view(torch.float32)


def _ceil_bf16(x):
    """The smallest bf16 that is not below x (64 bits, not negative)."""
    f = x.float()
    f = torch.where(f.double() < x, torch.nextafter(f, torch.full_like(f, math.inf)), f)
    bits = f.view(torch.int32)
    return ((bits + 0xffff) & -0x10000).view(torch.float32)


def _quantize4(x):
    """x [..., d] to codes [..., d / 32, 32], s and m [..., d / 32].  Which code
    is nearest is decided in 64 bits."""
    x = x.float().unflatten(-1, (-1, 32))
    m = _floor_bf16(x.amin(-1))
    s = _ceil_bf16((x.amax(-1).double() - m.double()) / torch.full((), 15.0, dtype=torch.float64, device=x.device))
    v = (x.double() - m.double()[..., None]) / torch.where(s > 0, s, 1.0).double()[..., None]
    return torch.floor(v + 0.5).clamp(0, 15).int(), s, m


def _places(tables, lengths, starts, nt, page, hkv, d):
    """Where the last tokens of each sequence stand in a cache's words: for each
    packed token and head the block's first word, and u, h, i of the token."""
    t = torch.arange(nt, device=tables.device)
    seq = torch.searchsorted(starts, t, right=True) - 1
    pos = lengths[seq].long() - starts[seq + 1].long() + t
    p = tables[seq, pos // page].long()
    block = (p[:, None] * hkv + torch.arange(hkv, device=p.device)) * (page // 32) + (pos % page // 32)[:, None]
    r = pos % 32
    return block * (10 * d), r // 16, r % 16 // 4, r % 4


def _word_places(first, u, h, i, d):
    """Words of the keys' codes [nt][hkv][d / 32][4], half words of the values'
    [nt][hkv][d / 64][16] and words of the keys' scales [nt][hkv][d / 32]."""
    dev, g = first.device, d // 32
    grp, e = torch.arange(g, device=dev), torch.arange(4, device=dev)
    w = u[:, None] * g + grp
    k = ((w // 4 * 64 + (4 * h + i)[:, None])[:, :, None] + e * 16) * 4 + (w % 4)[:, :, None]
    n, l16 = torch.arange(d // 64, device=dev), torch.arange(16, device=dev)
    w = (u * 2 + i // 2)[:, None] * (d // 64) + n
    v = 4 * d + ((w // 4 * 64)[:, :, None] + (h * 16)[:, None, None] + l16) * 4 + (w % 4)[:, :, None]
    v = 2 * v + (i % 2)[:, None, None]
    sc = 8 * d + (h * 8 + u * 4 + i)[:, None] * g + grp
    return first[:, :, None, None] + k[:, None], 2 * first[:, :, None, None] + v[:, None], first[:, :, None] + sc[:, None]


def _scale_word(s, m):
    return ((s.view(torch.int32) >> 16) & 0xffff) | (m.view(torch.int32) & -0x10000)


def _write_plain(k, v, pages, tables, lengths, starts, page):
    nt, hkv, d = k.shape
    kw, vh, sw = _word_places(*_places(tables, lengths, starts, nt, page, hkv, d), d)
    words, halves = pages.view(torch.int32).view(-1), pages.view(torch.int16).view(-1)
    b4 = 4 * torch.arange(4, device=k.device)
    at = torch.stack([b4, b4 + 16], 1)                                     # [b][a]
    c, s, m = _quantize4(k)
    words[kw] = (c.unflatten(-1, (4, 4, 2)).long() << at).sum((-1, -2)).int()
    words[sw] = _scale_word(s, m)
    c, s, m = _quantize4(v)
    halves[vh] = (c.flatten(-2).unflatten(-1, (d // 64, 4, 16)).long() << b4[:, None]).sum(-2).short()
    words[sw + d] = _scale_word(s, m)


def _scaled(codes, word):
    """The values that codes [..., d / 32, 32] and their scales' words stand for."""
    s, m = (word << 16).view(torch.float32), (word & -0x10000).view(torch.float32)
    return (codes.float() * s[..., None] + m[..., None]).flatten(-2)


def _read_plain(pages, tables, lengths, starts, nt, page, d):
    hkv = pages.shape[1]
    kw, vh, sw = _word_places(*_places(tables, lengths, starts, nt, page, hkv, d), d)
    words, halves = pages.view(torch.int32).view(-1), pages.view(torch.int16).view(-1)
    b4 = 4 * torch.arange(4, device=pages.device)
    at = torch.stack([b4, b4 + 16], 1)
    k = (words[kw][..., None, None] >> at) & 15                            # [nt][hkv][g][e][b][a]
    v = (halves[vh].int()[..., None, :] >> b4[:, None]) & 15               # [nt][hkv][n][b][l]
    return [_scaled(k.flatten(-3), words[sw]), _scaled(v.flatten(-3).unflatten(-1, (-1, 32)), words[sw + d])]


def _decoded(pages, tables, d):
    """Keys and values of whole sequences, [nseq][hkv][width * page][d]."""
    w = pages[tables.clamp(min=0).long()].view(torch.int32).unflatten(-1, (-1, 10 * d)).transpose(1, 2).flatten(2, 3)
    lead = list(range(w.dim() - 1))                                        # [nseq][hkv][blocks]
    g, n, b4 = d // 32, d // 64, 4 * torch.arange(4, device=pages.device)
    at = torch.stack([b4, b4 + 16], 1)
    perm = lambda x, *order: x.permute(lead + [len(lead) + o for o in order])  # noqa: E731
    k = perm(w[..., :4 * d].unflatten(-1, (-1, 4, 16, 4)), 0, 3, 1, 2)     # [w / 4][w % 4][e][l]
    k = perm(k.flatten(3, 4).unflatten(3, (2, g)), 0, 3, 1, 2)             # [u][l][g][e]
    k = ((k[..., None, None] >> at) & 15).flatten(-3).flatten(3, 4)        # [token][g][32]
    v = perm(w[..., 4 * d:8 * d].unflatten(-1, (-1, 4, 16, 4)), 0, 3, 1, 2).flatten(3, 4).unflatten(3, (2, 2, n))
    v = (v[..., None, None] >> at) & 15                                    # [u][i / 2][n][h][l][b][a]
    v = perm(v, 0, 3, 1, 6, 2, 5, 4).flatten(3, 6).flatten(4).unflatten(-1, (g, 32))
    sc = perm(w[..., 8 * d:].unflatten(-1, (2, 4, 2, 4, g)), 0, 2, 1, 3, 4).flatten(4, 6)  # [k, v][token][g]
    return [_scaled(c, x).flatten(2, 3) for c, x in ((k, sc[:, :, :, 0]), (v, sc[:, :, :, 1]))]


def _cached_plain(s):
    c = s["case"]
    nt, d = sum(_cache_lens(c)[0]), c["d"]
    if c["op"] == "write":
        _write_plain(s["k"], s["v"], s["pages"], s["tables"], s["lengths"], s["starts"], c["page"])
        return _read_plain(s["pages"], s["tables"], s["lengths"], s["starts"], nt, c["page"], d)
    k, v = _decoded(s["pages"], s["tables"], d)
    y = _attend_plain(_spread(s["q"], s["starts"], c["new"]), k, v, s["starts"][1:].long() - s["starts"][:-1].long(),
                      s["lengths"].long(), 1 / math.sqrt(d), True)
    return _packed(y, s["starts"], nt).to(TYPES[c["x"]])


# --- plain forms: pages ---------------------------------------------------------------------------------------------

def _held(s):
    """The pool's integers as a pass finds them: a pass changes its own copy."""
    c, held = s["case"], s["held"].clone()
    n = c["rows"] * c["width"]
    return held[:n].view(c["rows"], c["width"]), held[n:n + c["rows"]], held[n + c["rows"]:]


def _release_plain(tables, lengths, refs, rows):
    p = tables[rows].flatten()
    refs.index_add_(0, p.clamp(min=0), -(p >= 0).int())
    tables[rows] = -1
    lengths[rows] = 0


def _give(refs, need):
    """For each need in order the lowest free page, or -1; and how many get none."""
    order = torch.sort((refs > 0).int(), stable=True)[1]
    rank = need.int().cumsum(0)
    ok = need & (rank <= (refs <= 0).sum())
    p = torch.where(ok, order[(rank - 1).clamp(0, refs.shape[0] - 1)], -1)
    refs.index_add_(0, p.clamp(min=0), ok.int())
    return p.int(), (need & ~ok).sum().int()


def _fork_plain(pages, tables, lengths, refs, parents, children, page):
    _release_plain(tables, lengths, refs, children)
    row, n = tables[parents], lengths[parents]
    full = n // page
    col = torch.arange(tables.shape[1], device=row.device)
    share = (col < full[:, None]) & (row >= 0)
    refs.index_add_(0, row.clamp(min=0).flatten(), share.flatten().int())
    last = (col == full[:, None]) & (n % page > 0)[:, None] & (row >= 0)
    src = torch.where(last, row, -1).amax(1)
    dst, missing = _give(refs, src >= 0)
    tables[children] = torch.where(share, row, torch.where(last, dst[:, None], -1))
    lengths[children] = n
    moved = torch.nonzero(dst >= 0)[:, 0]
    pages[dst[moved].long()] = pages[src[moved].long()]
    return missing


def _take_plain(tables, lengths, refs, page):
    col = torch.arange(tables.shape[1], device=tables.device)
    need = (col < ((lengths + page - 1) // page)[:, None]) & (tables < 0)
    p, missing = _give(refs, need.flatten())
    tables.copy_(torch.where(need, p.view(tables.shape), tables))
    return missing


def _compact_plain(pages, tables, refs):
    live = refs > 0
    used = live.sum()
    at = torch.arange(refs.shape[0], device=refs.device)
    high, hole = torch.nonzero(live & (at >= used))[:, 0], torch.nonzero(~live & (at < used))[:, 0]
    pages[hole] = pages[high]
    refs[hole] = refs[high]
    refs[high] = 0
    at[high] = hole
    tables.copy_(torch.where(tables >= 0, at[tables.clamp(min=0).long()].int(), tables))
    return used.int()


def _pages_plain(s):
    c = s["case"]
    tables, lengths, refs = _held(s)
    out = [s["pages"], tables, lengths, refs]
    if s["rows"].numel():
        _release_plain(tables, lengths, refs, s["rows"])
    if s["parents"].numel():
        out.append(_fork_plain(s["pages"], tables, lengths, refs, s["parents"], s["children"], s["page"]))
    if c["grow"]:
        lengths += s["grown"]
        out.append(_take_plain(tables, lengths, refs, s["page"]))
    if s["src"].numel():
        s["pages"][s["dst"].long()] = s["pages"][s["src"].long()]
    if c["compact"]:
        out.append(_compact_plain(s["pages"], tables, refs))
    return out


def _plain(s):
    op = s["case"]["op"]
    return _prompt_plain(s) if op == "prompt" else _pages_plain(s) if op == "pages" else _cached_plain(s)


# --- the package's calls --------------------------------------------------------------------------------------------

def _own(s):
    import quant_integer_gemm_amd as qig
    c = s["case"]
    if c["op"] == "prompt":
        return qig.attend_prompt(s["q"], s["k"], s["v"], s["starts"], s["k_starts"], causal=c["causal"])
    if c["op"] == "write":
        qig.write_kv4(s["k"], s["v"], s["pages"], s["tables"], s["lengths"], s["starts"])
        return list(qig.read_kv4(s["pages"], s["tables"], s["lengths"], c["d"], s["starts"], s["k"].shape[0]))
    if c["op"] == "attend":
        return qig.attend_kv4(s["q"], s["pages"], s["tables"], s["lengths"], s["starts"],
                              ws=qig.workspace(s["q"].device))
    tables, lengths, refs = _held(s)
    out = [s["pages"], tables, lengths, refs]
    if s["rows"].numel():
        qig.free_pages(tables, lengths, refs, s["rows"])
    if s["parents"].numel():
        out.append(qig.fork_pages(s["pages"], tables, lengths, refs, s["parents"], s["children"], s["page"])[0])
    if c["grow"]:
        lengths += s["grown"]
        out.append(qig.take_pages(tables, lengths, refs, s["page"])[0])
    if s["src"].numel():
        qig.copy_pages(s["pages"], s["src"], s["dst"])
    if c["compact"]:
        out.append(qig.compact_pages(s["pages"], tables, refs)[0])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# --- the work of a pass ---------------------------------------------------------------------------------------------

def _pairs(nq, nk, causal):
    """(query, key) pairs that are seen."""
    return nq * (nk - nq) + nq * (nq + 1) // 2 if causal else nq * nk


def work(case):
    c, op = case, case["op"]
    if op == "pages":
        entries = c["rows"] * c["width"] + c["rows"] + c["npages"]
        moved = c["forks"] + c["copies"]
        if c["compact"]:   # of the pages still in use, scattered evenly, those behind the front that they will fill
            used = 0.9 * c["rows"] * (c["width"] - 1) / math.log(c["width"])
            used = min(0.8 * c["npages"], used) * (1 - c["frees"] / (0.9 * c["rows"]))
            moved += int(used * (1 - used / c["npages"]))
        return {"bytes": 8 * entries + 8 * moved * c["words"], "flops": entries}
    d, hq, hkv = c["d"], c["hq"], c["hkv"]
    if op == "prompt":
        n, nk = _prompt_lens(c)
        return {"bytes": 2 * d * BYTES[c["x"]] * (hq * sum(n) + hkv * sum(nk)),
                "flops": 4 * hq * d * sum(_pairs(a, b, c["causal"]) for a, b in zip(n, nk))}
    n, lens = _cache_lens(c)
    if op == "write":
        return {"bytes": int(2 * sum(n) * hkv * d * (BYTES[c["x"]] + 0.625 + 0.625 + 4)), "flops": 12 * sum(n) * hkv * d}
    return {"bytes": int(2 * sum(n) * hq * d * BYTES[c["x"]] + 1.25 * sum(lens) * hkv * d),
            "flops": 4 * hq * d * sum(_pairs(a, b, True) for a, b in zip(n, lens))}


# --- 64 bits, from the definitions ----------------------------------------------------------------------------------

def _exact_attention(q, k, v, causal):
    """One sequence: q [n][hq][d], k and v [nk][hkv][d] in 64 bits, some rows of
    queries at a time."""
    n, hq, d = q.shape
    nk, hkv, _ = k.shape
    y = torch.zeros_like(q)
    size = max(1, (1 << 28) // max(1, nk * hq))
    kt, vt = k.permute(1, 2, 0).contiguous(), v.transpose(0, 1).contiguous()
    for a in range(0, n, size):
        rows = q[a:a + size]
        m = rows.shape[0]
        x = rows.view(m, hkv, hq // hkv, d).permute(1, 0, 2, 3).reshape(hkv, -1, d)
        s = torch.bmm(x, kt).view(hkv, m, hq // hkv, nk) * d ** -0.5
        if causal:
            hidden = torch.ones((m, nk), dtype=torch.bool, device=q.device).triu(nk - n + a + 1)
            s[hidden[None, :, None, :].expand_as(s)] = -math.inf
        p = torch.softmax(s, -1).nan_to_num(0.0).view(hkv, -1, nk)
        y[a:a + size] = torch.bmm(p, vt).view(hkv, m, hq // hkv, d).permute(1, 0, 2, 3).reshape(m, hq, d)
    return y


def _exact_4bit(x):
    """The values that 4 bits leave of x, from the definition."""
    x = x.to(torch.float64)
    parts = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))

    def near(t, rounded):
        step = torch.frexp(t)[1].long() - 8                                # of 8 significant bits
        unit = ((step + 1023) << 52).view(torch.float64)                   # 2^step: its exponent's bits
        return rounded(t / unit) * unit

    m = near(parts.min(-1, keepdim=True).values, torch.floor)
    s = near((parts.max(-1, keepdim=True).values - m) / torch.full_like(m, 15.0), torch.ceil)   # a true division
    c = torch.where(s > 0, (parts - m) / s, torch.zeros_like(parts)).add(0.5).floor().clamp(max=15)
    return (m + s * c).reshape(x.shape)


def _exact_maps(d):
    """Bit positions in a block of every (token, channel), and the scale's bit
    positions, by the layout's text."""
    k, v, s = [], [], []
    for t in range(32):
        u, h, i = t // 16, t % 16 // 4, t % 4
        for ch in range(d):
            g, e, b, a = ch // 32, ch % 32 // 8, ch % 8 // 2, ch % 2
            w = u * (d // 32) + g
            k.append(32 * (((w // 4) * 64 + e * 16 + 4 * h + i) * 4 + w % 4) + 16 * a + 4 * b)
            n, b, l16 = ch // 64, ch // 16 % 4, ch % 16
            w = (2 * u + i // 2) * (d // 64) + n
            v.append(32 * (4 * d + ((w // 4) * 64 + h * 16 + l16) * 4 + w % 4) + 16 * (i % 2) + 4 * b)
            s.append(32 * (8 * d + (h * 8 + u * 4 + i) * (d // 32) + g))
    return [torch.tensor(x, device="cuda").view(32, d) for x in (k, v, s)]


def _exact_cached(pages, row, length, page, d, maps):
    """Keys and values [length][hkv][d] of one sequence in 64 bits."""
    hkv = pages.shape[1]
    blocks = pages[row[:(length + page - 1) // page].long()].view(-1, hkv, page // 32, 40 * d)
    at_k, at_v, at_s = maps

    def one(at, more):
        codes = (blocks[..., at // 8] >> (at % 8).to(torch.uint8)) & 15
        half = lambda o: (blocks[..., at_s // 8 + more + o].to(torch.int32) << 16  # noqa: E731
                          | blocks[..., at_s // 8 + more + o + 1].to(torch.int32) << 24).view(torch.float32)
        x = half(0).double() * codes.double() + half(2).double()           # [pages][hkv][blocks][32][d]
        return x.permute(0, 2, 3, 1, 4).reshape(-1, hkv, d)[:length]

    return one(at_k, 0), one(at_v, 4 * d)


def exact(case, seed):
    c = case
    if c["op"] == "pages":
        return None
    s = prepare(case, seed)
    if c["op"] == "write":
        return [_exact_4bit(s["k"]), _exact_4bit(s["v"])]
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = s["starts"].tolist()
    if c["op"] == "prompt":
        kat = s["k_starts"].tolist()
        for a, b, ka, kb in zip(at, at[1:], kat, kat[1:]):
            y[a:b] = _exact_attention(s["q"][a:b].double(), s["k"][ka:kb].double(), s["v"][ka:kb].double(), c["causal"])
        return y
    maps = _exact_maps(c["d"])
    for i, (a, b) in enumerate(zip(at, at[1:])):
        k, v = _exact_cached(s["pages"], s["tables"][i], int(s["lengths"][i]), c["page"], c["d"], maps)
        y[a:b] = _exact_attention(s["q"][a:b].double(), k, v, True)
    return y
