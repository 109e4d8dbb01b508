"""The 8-bit paged cache, the attention over it and the adapters in 64 bits on
the CPU, from their definitions, and how far the kernels may be from them."""
import numpy as np
import torch

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64


class Batch:
    """Sequences with ``new[s]`` new tokens after ``before[s]`` cached ones, on
    shuffled pages; ``extra`` rows of the packed buffers belong to no sequence."""

    def __init__(self, new, before, P, heads, D, seed=0, extra=0, spare=2, width=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.before, self.P, self.heads, self.D = list(new), list(before), P, heads, D
        self.S, self.T = len(new), sum(new) + extra
        total = [n + c for n, c in zip(new, before)]
        each = [-(-t // P) for t in total]
        self.width = max([width, 1] + each)
        self.pages = sum(each) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((self.S, self.width), -7, dtype=torch.int32)
        at = 0
        for s, n in enumerate(each):
            for i in range(n):
                self.table[s, i] = order[at]
                at += 1
        self.starts = torch.zeros(self.S + 1, dtype=torch.int32)
        self.starts[1:] = torch.tensor(list(new), dtype=torch.int32).cumsum(0)
        self.lengths = torch.tensor(total, dtype=torch.int32)
        self.k_pages = torch.randint(-128, 128, (self.pages, heads, P, D), generator=g, dtype=torch.int8)
        self.v_pages = torch.randint(-128, 128, (self.pages, heads, D, P), generator=g, dtype=torch.int8)
        self.k_scales = torch.exp2(torch.randint(-8, -4, (self.pages, heads), generator=g).float())
        self.v_scales = torch.exp2(torch.randint(-9, -3, (self.pages, heads), generator=g).float())

    def index(self):
        return self.starts, self.lengths, self.table

    def cache(self):
        return self.k_pages, self.v_pages, self.k_scales, self.v_scales

    def cuda(self):
        """(starts, lengths, table, k_pages, v_pages, k_scales, v_scales) on the GPU."""
        return [t.cuda() for t in self.index() + self.cache()]


def rotate(x, cos, sin, interleaved):
    """x [..., D] in 64 bits, cos and sin [rot / 2] of its position."""
    x = x.double().clone()
    half = cos.shape[-1]
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c, s = cos[..., j].double(), sin[..., j].double()
        p, q = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = p * c - q * s, q * c + p * s
    return x


def fitting_scale(values, scale):
    """The smallest power of two from ``scale`` (0: none yet) up under which all
    values lie in -128 .. 128; NaN where one is not finite."""
    if np.isnan(scale) or not bool(torch.isfinite(values).all()):
        return float("nan")
    hi, lo = float(values.max()), float(values.min())
    if scale == 0 and (hi or lo):
        scale = 2.0 ** -126
    while scale and not (-128 * scale <= lo and hi < 128 * scale):
        scale *= 2
    return scale


def append(b, k, v, cos, sin, q=None, interleaved=False):
    """Stores the new tokens into b's cache; returns the rotated q in 64 bits (NaN
    in rows that get none)."""
    out = None if q is None else torch.full(q.shape, float("nan"), dtype=F64)
    for s in range(b.S):
        t0, n = int(b.starts[s]), int(b.starts[s + 1] - b.starts[s])
        start = int(b.lengths[s]) - n
        pages = {}
        for i in range(n):
            pos = start + i
            if pos < 0 or pos >= b.width * b.P:
                continue
            kk, vv = k[t0 + i].double(), v[t0 + i].double()
            qq = None if q is None else q[t0 + i].double()
            if cos is not None:
                kk = rotate(kk, cos[pos], sin[pos], interleaved)
                qq = qq if q is None else rotate(qq, cos[pos], sin[pos], interleaved)
            if q is not None:
                out[t0 + i] = qq
            pages.setdefault(pos // b.P, []).append((pos % b.P, kk, vv))
        for index, tokens in pages.items():
            p = int(b.table[s, index])
            if not 0 <= p < b.pages:
                continue
            offs = [t[0] for t in tokens]
            first = min(offs)
            for h in range(b.heads):
                for which, scales in ((1, b.k_scales), (2, b.v_scales)):
                    vals = torch.stack([t[which][h] for t in tokens])
                    ints = b.k_pages[p, h] if which == 1 else b.v_pages[p, h].t()
                    old = float(scales[p, h]) if first else 0.0
                    new = fitting_scale(vals, old)
                    if old and not np.isnan(new):
                        ints[:first] = torch.floor(ints[:first].double() * (old / new)).to(torch.int8)
                    if np.isnan(new):
                        ints[offs] = 0
                    else:
                        ints[offs] = torch.floor(vals / (new or 1.0)).to(torch.int8)
                    scales[p, h] = new
    return out


def keys_of(b, s, h, upto):
    """Keys and values of positions 0 .. upto - 1 in 64 bits, the value integers
    (with their half) and scales, and which positions hold a token."""
    n = min(upto, b.width * b.P)
    k, v = torch.zeros(upto, b.D, dtype=F64), torch.zeros(upto, b.D, dtype=F64)
    held, vs = torch.zeros(upto, dtype=torch.bool), torch.zeros(upto, dtype=F64)
    for i in range(-(-n // b.P)):
        p = int(b.table[s, i])
        if not 0 <= p < b.pages:
            continue
        m = min(b.P, n - i * b.P)
        at = slice(i * b.P, i * b.P + m)
        k[at] = (b.k_pages[p, h, :m].double() + 0.5) * float(b.k_scales[p, h])
        v[at] = (b.v_pages[p, h, :, :m].t().double() + 0.5) * float(b.v_scales[p, h])
        vs[at] = float(b.v_scales[p, h])
        held[at] = True
    return k, v, vs, held


def attention(b, q, scale):
    """Rows [T][heads][D] in 64 bits, and how far the kernels' may be from them
    before their last rounding.

    Scores: the query's integers are off by 2^-22 of its largest element at
    most; the sum of their products, its factor and the exponential by 16 steps
    of 2^-24 of the sum of the products' magnitudes, and of the largest score.
    A score off by d moves a weight by 2 d relative at most.
    Weights: 16 bits against the unit's largest weight times value scale
    (2^-16 of it each, an integer of 128 at most), or 2^-11 of each and 2^-24 of
    the row's largest where they are held in fp16.
    Sums: a step of 2^-24 for every unit of 64 keys and 64 more, of the sum of the
    magnitudes.
    """
    T, hq, D = q.shape
    G = hq // b.heads
    out = torch.full(q.shape, float("nan"), dtype=F64)
    tol = torch.zeros(q.shape, dtype=F64)
    for s in range(b.S):
        t0, n = int(b.starts[s]), int(b.starts[s + 1] - b.starts[s])
        length = int(b.lengths[s])
        upto = min(max(length, 0), b.width * b.P)
        for h in range(b.heads if n else 0):
            k, v, vs, held = keys_of(b, s, h, upto)
            rows = q[t0:t0 + n, h * G:(h + 1) * G].double().reshape(n * G, D)
            last = (length - n + torch.arange(n)).repeat_interleave(G)
            seen = held[None] & (torch.arange(upto)[None] <= last[:, None])
            some = seen.any(dim=1)
            y = torch.zeros(n * G, D, dtype=F64)
            e = torch.zeros(n * G, D, dtype=F64)
            if bool(some.any()):
                z = (rows @ k.t() * scale).masked_fill(~seen, float("-inf"))
                w = torch.softmax(z[some], dim=1)
                y[some] = w @ v
                m = seen[some]
                kmag = k.abs().sum(dim=1)[None].masked_fill(~m, 0)
                mag = abs(scale) * (rows[some].abs() @ k.abs().t()).masked_fill(~m, 0)
                largest = z[some].masked_fill(~m, 0).abs().amax(dim=1)
                d = abs(scale) * 2.0 ** -22 * rows[some].abs().amax(dim=1) * kmag.amax(dim=1)
                d = d + 16 * 2.0 ** -24 * (mag.amax(dim=1) + largest)
                size = w @ v.abs()
                moved = 2 * d[:, None] * (size + y[some].abs())
                pad = -upto % 64
                ws = torch.nn.functional.pad(w * vs[None], (0, pad)).reshape(w.shape[0], -1, 64)
                held16 = 2.0 ** -16 * 128 * 64 * ws.amax(dim=2).sum(dim=1)[:, None]
                total = (m * vs[None]).sum(dim=1)[:, None]
                heldf = 2.0 ** -11 * size + 2.0 ** -24 * 128 * w.amax(dim=1)[:, None] * total
                sums = (ws.shape[1] + 64) * 2.0 ** -24 * 2 * (size + 128 * (w @ vs)[:, None])
                e[some] = moved + torch.maximum(held16.expand_as(size), heldf) + sums
            out[t0:t0 + n, h * G:(h + 1) * G] = y.reshape(n, G, D)
            tol[t0:t0 + n, h * G:(h + 1) * G] = e.reshape(n, G, D)
    return out, tol


def check_rows(got, want, tol, dtype):
    """got (CPU, dtype) against want within tol and one rounding to dtype."""
    x, info = got.double(), torch.finfo(dtype)
    nan = torch.isnan(want)
    assert bool((torch.isnan(x) == nan).all())
    rounding = info.eps / 2 * want.abs() + info.smallest_normal * info.eps
    bad = ((x - want).abs() > tol * (1 + info.eps) + rounding) & ~nan
    assert not bool(bad.any()), "%d of %d off, worst %.3g of %.3g allowed" % (
        int(bad.sum()), bad.numel(), float((x - want).abs()[bad].max()), float((tol + rounding)[bad].max()))


def lora(x, ids, A, B, scaling, base):
    """out in 64 bits, and how far the kernels' may be from it before their last
    rounding: K + 64 steps of 2^-24 in A x (and the scaling), the two pieces that
    hold it (2^-16 of a bf16 sum; 2^-22 of an fp16 one and 2^-25 of the row's
    largest), 2 R + 64 steps in the second product and the sum with the base."""
    m, K = x.shape
    n, R, _ = A.shape
    y = torch.zeros(m, B.shape[1], dtype=F64) if base is None else base.double().clone()
    tol = torch.zeros_like(y)
    for r in range(m):
        a = int(ids[r])
        if not 0 <= a < n:
            continue
        s = 1.0 if scaling is None else float(scaling[a])
        Ad, Bd, xd = A[a].double(), B[a].double(), x[r].double()
        t = Ad @ xd * s
        mag = (Ad.abs() @ xd.abs()) * abs(s)
        dt = (K + 64) * 2.0 ** -24 * mag
        if x.dtype == BF16:
            dt = dt + 2.0 ** -16 * t.abs()
        else:
            dt = dt + 2.0 ** -22 * t.abs() + 2.0 ** -24 * float(t.abs().max())
        d = Bd @ t
        tol[r] = Bd.abs() @ dt + (2 * R + 64) * 2.0 ** -24 * (Bd.abs() @ t.abs()) + 2.0 ** -23 * (y[r].abs() + d.abs())
        y[r] += d
    return y, tol
