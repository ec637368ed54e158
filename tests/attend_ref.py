"""Plain 64-bit forms of the attention operators, the 4-bit cache and its pages, on
the CPU, written from the definitions in include/qig.h, and how far a result
may be from them."""
import numpy as np
import torch

# half a step of each type, relative to the value, and half of its smallest step
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FLOOR = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
E32 = 2.0 ** -24


def attention(q, k, v, nq_total, pos, scale, seen_pages=None):
    """(y, sum p |v|, largest sum |q k| scale) of queries q [n][hq][d] at the
    positions pos over keys k and values v [nk][hkv][d]; query i sees the keys up to
    pos[i] (seen_pages: of them, those that are true).  All in 64 bits."""
    q, k, v = (t.double().cpu() for t in (q, k, v))
    n, hq, d = q.shape
    nk, hkv, _ = k.shape
    k, v = (t.repeat_interleave(hq // hkv, 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, k) * scale
    big = torch.einsum("ihd,jhd->hij", q.abs().nan_to_num(0, 0, 0), k.abs().nan_to_num(0, 0, 0)) * scale
    see = torch.arange(nk)[None, :] <= torch.as_tensor(pos)[:, None]
    if seen_pages is not None:
        see = see & seen_pages[None, :]
    s = s.masked_fill(~see[None], -np.inf)
    big = big.masked_fill(~see[None], 0.0)
    top = s.amax(2, keepdim=True) if nk else torch.zeros((hq, n, 1), dtype=torch.float64)
    top = torch.where(top == -np.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(2, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    # what a query does not see has no effect, whatever it holds
    y = torch.zeros((n, hq, d), dtype=torch.float64)
    mag = torch.zeros((n, hq, d), dtype=torch.float64)
    for i in range(n):
        j = torch.nonzero(see[i])[:, 0]
        y[i] = torch.einsum("hj,jhd->hd", p[:, i, j], v[j])
        mag[i] = torch.einsum("hj,jhd->hd", p[:, i, j], v[j].abs())
    amax = big.amax(2).T[:, :, None] if nk else torch.zeros((n, hq, 1), dtype=torch.float64)
    return y, mag, amax


def allowance(y, mag, amax, d, nk, p_step, ytype):
    """Scores: a dot product of d terms is off by at most (d + 3) half steps of fp32
    relative to its terms' sizes (its sum, the scale's rounding and two of the
    exponent's), and p by that factor; so is the sum of the p's.  The power itself, l's and
    O's sums over nk keys, their corrections (one a step of 32 keys at most, in each of
    up to four parts and their join) and the division: below 3 nk + 16 more.  p_step: half a
    step of what p is rounded to for the second product.  y: one rounding."""
    rel = 2 * ((d + 3) * E32 * amax) + (3 * nk + 16) * E32 + p_step
    err = mag * rel * 1.0001
    return err + EPS[ytype] * (y.abs() + err) + FLOOR[ytype]


def check(got, y, allow, what=""):
    got = got.double().cpu()
    bad = torch.isnan(y)
    assert torch.equal(torch.isnan(got), bad), f"{what}: NaN in other places"
    over = ((got - y).abs() / allow)[~bad]
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowance"
    return worst


# --- the 4-bit cache ---------------------------------------------------------------------------------------------

def bf16_floor(x):
    """The largest bf16 <= x (fp32, finite), as fp32: by stepping from the nearest."""
    n = torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)
    down = torch.nextafter(n, torch.tensor(-np.inf, dtype=torch.bfloat16))
    return torch.where(n.double() > torch.from_numpy(x.astype(np.float64)), down, n).float().numpy()


def bf16_ceil(x):
    """The smallest bf16 >= x (64 bits)."""
    n = torch.from_numpy(x).to(torch.bfloat16)
    up = torch.nextafter(n, torch.tensor(np.inf, dtype=torch.bfloat16))
    down = torch.nextafter(n, torch.tensor(-np.inf, dtype=torch.bfloat16))
    at = torch.from_numpy(x)
    n = torch.where(n.double() < at, up, n)
    return torch.where((down.double() >= at), down, n).float().numpy()


def quantize4(x):
    """codes [..., d / 32, 32], s and m [..., d / 32] of finite x [..., d]."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32)).astype(np.float64)
    m = bf16_floor(g.min(-1).astype(np.float32)).astype(np.float64)
    s = bf16_ceil((g.max(-1) - m) / 15.0).astype(np.float64)
    safe = np.where(s > 0, s, 1.0)
    c = np.floor((g - m[..., None]) / safe[..., None] + 0.5)
    return np.where(s[..., None] > 0, np.clip(c, 0, 15), 0).astype(np.uint8), s.astype(np.float32), m.astype(np.float32)


def values4(c, s, m):
    """What they stand for, in fp32: one rounding."""
    return (m[..., None].astype(np.float64) + s[..., None].astype(np.float64) * c).astype(np.float32).reshape(
        c.shape[:-2] + (c.shape[-2] * 32,))


def stands_for(x):
    return values4(*quantize4(x))


def block_bytes(kc, ks, km, vc, vs, vm):
    """The 40 d bytes of a block from the codes [32][d / 32][32] and scales [32][d / 32]
    of its keys and values, by the header's text."""
    d = kc.shape[1] * 32
    words = np.zeros(10 * d, dtype=np.uint32)

    def pair(s, m):
        s16 = s.astype(np.float32).view(np.uint32) >> 16
        return s16 | (m.astype(np.float32).view(np.uint32) & 0xffff0000)

    kw, vw = pair(ks, km), pair(vs, vm)
    kc, vc = kc.reshape(32, d), vc.reshape(32, d)
    for t in range(32):
        u, h, i = t // 16, t % 16 // 4, t % 4
        for ch in range(d):
            g, e, b, a = ch // 32, ch % 32 // 8, ch % 8 // 2, ch % 2
            w = u * d // 32 + g
            words[((w // 4) * 64 + e * 16 + 4 * h + i) * 4 + w % 4] |= np.uint32(int(kc[t, ch]) << (16 * a + 4 * b))
            n, b, l16 = ch // 64, ch // 16 % 4, ch % 16
            w = (2 * u + i // 2) * d // 64 + n
            words[4 * d + ((w // 4) * 64 + h * 16 + l16) * 4 + w % 4] |= np.uint32(int(vc[t, ch]) << (16 * (i % 2) + 4 * b))
        for g in range(d // 32):
            words[8 * d + (h * 8 + u * 4 + i) * d // 32 + g] = kw[t, g]
            words[9 * d + (h * 8 + u * 4 + i) * d // 32 + g] = vw[t, g]
    return words.view(np.uint8)


def kv4_allowance(q, mag, amax, amp, d, nk, qtype, ytype, smax):
    """As allowance(), for attend_kv4.  amax: the largest sum over channels of |q| (|m| +
    s c) scale; mag: sum p (|m| + s c).  A score has besides (d + 3) the group sums' d / 16
    products and sums; fp32 queries keep 22 bits (2^-22), and what falls below f16's
    smallest step is 2^-39 of the row's largest |q| (amp: that times the sum of s c
    scale).  p s: 2^-11, or 2^-22 in two parts, and half of f16's smallest step, 2^-25 of
    2^(6 - E): below 2^-30 of the largest scale a token, times code 15."""
    score = (d + 3 + d // 16) * E32 * amax + (2.0 ** -22 * amax if qtype == torch.float32 else 0) + 2.0 ** -39 * amp
    step = 2.0 ** -11 if ytype == torch.bfloat16 else 2.0 ** -22
    err = mag * (2 * score + (3 * nk + 32) * E32 + step) * 1.0001 + nk * 15 * 2.0 ** -30 * smax
    return lambda y: err + EPS[ytype] * (y.abs() + err) + FLOOR[ytype]


# --- pages -------------------------------------------------------------------------------------------------------

class Pool:
    """tables, lengths and refs as lists, with the pages' operators one step after the other."""

    def __init__(self, tables, lengths, refs):
        self.t, self.len, self.refs = [list(r) for r in tables], list(lengths), list(refs)

    def ok(self, p):
        return 0 <= p < len(self.refs)

    def free_list(self):
        return [p for p, r in enumerate(self.refs) if r <= 0]

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.t):
                for c, p in enumerate(self.t[r]):
                    if self.ok(p) and self.refs[p] > 0:
                        self.refs[p] -= 1
                    self.t[r][c] = -1
                self.len[r] = 0

    def take(self, page):
        free, missing = self.free_list(), 0
        for r, n in enumerate(self.len):
            n = max(0, -(-n // page))
            for c in range(min(n, len(self.t[r]))):
                if not self.ok(self.t[r][c]):
                    self.t[r][c] = -1
                    if free:
                        self.t[r][c] = free.pop(0)
                        self.refs[self.t[r][c]] = 1
                    else:
                        missing += 1
        return missing

    def fork(self, parents, children, page):
        """(missing, [(src, dst)])"""
        n = len(self.t)
        good = [i for i, (a, b) in enumerate(zip(parents, children))
                if 0 <= a < n and 0 <= b < n and a not in children and b not in children[i + 1:]]
        self.free([children[i] for i in good])
        copies, wait = [], []
        for i in good:
            a, b = parents[i], children[i]
            length = self.len[a]
            full = max(0, length) // page
            for c in range(min(full, len(self.t[a]))):
                if self.ok(self.t[a][c]):
                    self.t[b][c] = self.t[a][c]
                    self.refs[self.t[a][c]] += 1
            self.len[b] = length
            if length > 0 and length % page and full < len(self.t[a]) and self.ok(self.t[a][full]):
                wait.append((self.t[a][full], b, full))
        free, missing = self.free_list(), 0
        for src, b, c in wait:
            if free:
                dst = free.pop(0)
                self.refs[dst] = 1
                self.t[b][c] = dst
                copies.append((src, dst))
            else:
                missing += 1
        return missing, copies

    def compact(self):
        """(used, to, [(src, dst)])"""
        used = sum(r > 0 for r in self.refs)
        high = [p for p, r in enumerate(self.refs) if r > 0 and p >= used]
        hole = [p for p, r in enumerate(self.refs) if r <= 0 and p < used]
        to = list(range(len(self.refs)))
        for a, b in zip(high, hole):
            to[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.t = [[to[p] if self.ok(p) else p for p in row] for row in self.t]
        return used, to, list(zip(high, hole))
