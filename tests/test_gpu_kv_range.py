"""Calls at the ends of what the cache, the attention over it and the adapters
take: scores, scales and lengths that lie far apart, values next to a type's
largest and smallest."""
import math

import pytest
import torch

import block_wise_int4_matmulnbits_amd as mnb
from tests import gpu_util as G
from tests import kv_ref as R
from tests import test_gpu_append as APP
from tests import test_gpu_attention as ATT

pytestmark = pytest.mark.gpu

F16, BF16, F64 = torch.float16, torch.bfloat16, torch.float64


def _few_rows(b, q, scale):
    """Rows in 64 bits, and how far those of a sequence of few rows may be from
    them before their last rounding.

    As R.attention's, with the terms that belong to few rows alone: a score is off
    by 2^-22 of its query's largest element and 16 steps of 2^-24 of the products'
    magnitudes and of the largest score, a weight by twice that relative; each
    weight is off by 1 / 65024 of the largest weight times value scale of its 64
    keys, an integer of 128 at most, and what lies below 2^-126 of the row's
    largest may count as zero; a sum by 2^-24 for each unit of 64 keys and 64
    more, of its magnitudes, and by fp32's smallest step for each unit.
    """
    T, hq, D = q.shape
    G_ = hq // b.heads
    out, tol = torch.full(q.shape, float("nan"), dtype=F64), torch.zeros(q.shape, dtype=F64)
    for s in range(b.S):
        t0, n, length = int(b.starts[s]), int(b.starts[s + 1] - b.starts[s]), int(b.lengths[s])
        for h in range(b.heads):
            k, v, vs, held = R.keys_of(b, s, h, length)
            for i in range(n * G_):
                t, head = t0 + i // G_, h * G_ + i % G_
                m = held & (torch.arange(length) <= length - n + i // G_)
                x = q[t, head].double()
                z = (k @ x * scale)[m]
                w = torch.softmax(z, dim=0)
                y = w @ v[m]
                mag = abs(scale) * (k.abs() @ x.abs())[m]
                d = abs(scale) * 2.0 ** -22 * x.abs().max() * k[m].abs().sum(dim=1).max()
                d = d + 16 * 2.0 ** -24 * (mag.max() + z.abs().max())
                size = w @ v[m].abs()
                ws = torch.zeros(-(-length // 64) * 64, dtype=F64)
                ws[:length][m] = w * vs[m]
                held16 = 128 * 64 / 65024 * ws.reshape(-1, 64).amax(dim=1).sum()
                units = ws.numel() // 64
                sums = (units + 64) * 2.0 ** -24 * 2 * (size + 128 * (w @ vs[m])) + units * 2.0 ** -149
                below = 2.0 ** -126 * 128 * float(vs[m].sum())
                out[t, head], tol[t, head] = y, 2 * d * (size + y.abs()) + held16 + sums + below
    return out, tol


def _scored(lengths, P, D, scores, scales, seed=1, new=None):
    """Sequences whose page i scores scores[i % len] (within one) for a query of one
    at element 0 and zeros elsewhere, and has the value scale scales[i % len]; the
    other integers are random."""
    new = new or [1] * len(lengths)
    b = R.Batch(new, [n - m for n, m in zip(lengths, new)], P, 1, D, seed=seed)
    b.k_scales[:] = 2
    for s in range(b.S):
        for i in range(-(-int(b.lengths[s]) // P)):
            p = int(b.table[s, i])
            b.k_pages[p, :, :, 0] = round(scores[i % len(scores)] / 2)
            b.v_scales[p] = scales[i % len(scales)]
    return b


def _unit_queries(T, hq, D):
    q = torch.zeros(T, hq, D)
    q[:, :, 0] = 1
    return q.to(BF16)


@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("gap", [80, 100, 114, 120, 130, 160, 200])
def test_largest_score_on_a_page_of_zeros(P, gap):
    """A page of zeros holds the largest scores, the other pages of the unit score
    `gap` (log2) lower."""
    G.require_gpu()
    low = -round(gap * 0.6931471805599453)
    b = _scored([64, 64 + 16, 190], P, 64, (0, low, low - 3, low + 2), (0.0, 0.25, 2.0, 1.0))
    q = _unit_queries(3, 2, 64)
    got = ATT._call(b, q, scale=1.0)
    want, tol = _few_rows(b, q, 1.0)
    R.check_rows(got, want, tol, BF16)


@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("far", [(-126, -5, 120), (-126, 0, 80), (-126, -5, 160), (-126, 100, 118), (-100, 20, 114), (-20, 100, 90)])
def test_scores_and_value_scales_far_apart(P, far):
    """The largest score under a small value scale, and the other way round."""
    G.require_gpu()
    one, two, gap = far
    low = -round(gap * 0.6931471805599453)
    for scores, scales in (((0, low), (2.0 ** one, 2.0 ** two)), ((low, 0), (2.0 ** two, 2.0 ** one)),
                           ((0, low, low - 1), (2.0 ** one, 2.0 ** two, 0.0))):
        b = _scored([64, 100, 300], P, 64, scores, scales)
        q = _unit_queries(3, 2, 64)
        got = ATT._call(b, q, scale=1.0)
        want, tol = _few_rows(b, q, 1.0)
        R.check_rows(got, want, tol, BF16)


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("first", [0, 2, 4, 8])
@pytest.mark.parametrize("e", [-126, -122, -112])
def test_small_value_scales(e, first, P):
    """Value scales down to the smallest, behind a page of zeros whose scores are
    larger: what the weights leave of them keeps its bits."""
    G.require_gpu()
    ahead = 1 if P < 64 else 4         # units of 64 keys go to four waves in turn
    b = _scored([128, 333] if P < 64 else [512, 1111], P, 64, (0,) * ahead + (-first,) * (4 * ahead - ahead),
                (0.0,) * ahead + (2.0 ** e, 2.0 ** (e + 2), 2.0 ** e) * ahead)
    b.v_pages[:] = b.v_pages.abs().clamp(min=64, max=127)         # no sum is near zero
    q = _unit_queries(2, 2, 64)
    got = ATT._call(b, q, scale=1.0)
    want, tol = _few_rows(b, q, 1.0)
    R.check_rows(got, want, tol, BF16)


def test_value_scales_below_the_normal_range():
    """Scales under 2^-126 count for something between nothing and what they are."""
    G.require_gpu()
    for P in (16, 32, 64):
        for gap in (0, 10, 40):
            b = _scored([64, 200], P, 64, (0, -gap, -gap), (2.0 ** -130, 2.0 ** -124, 2.0 ** -149))
            q = _unit_queries(2, 2, 64)
            got = ATT._call(b, q, scale=1.0)
            with_them = _few_rows(b, q, 1.0)
            b.v_scales[b.v_scales < 2.0 ** -126] = 0
            without = _few_rows(b, q, 1.0)
            tol = torch.maximum(with_them[1], without[1]) + (with_them[0] - without[0]).abs() / 2
            R.check_rows(got, (with_them[0] + without[0]) / 2, tol, BF16)


@pytest.mark.parametrize("hq,new", [(16, 40), (64, 70)], ids=["shares", "tiles"])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("es", [(-5, -70, -126), (0, -80, -126), (100, 30, -40, -110), (-126, -60, 10, 90), (-126, 0),
                                (0, -126, 100), (-30, -126, -126, 60)], ids=str)
def test_value_scales_fall_and_rise(es, P, hq, new):
    """Tiles: value scales that fall and rise by 2^200 in all, rows that see the
    first of them only."""
    G.require_gpu()
    b = _scored([900], P, 64, (0, 1, -1, 0, 2), tuple(2.0 ** e for e in es), new=[new])
    for first in (0, 64):
        if first:                  # rows that begin with the sequence
            b = _scored([new], P, 64, (0, 1, -1, 0, 2), tuple(2.0 ** e for e in es), new=[new])
        ATT._check(b, ATT._queries(new, hq, 64, BF16, 3, 0.125), scale=0.02)


def test_small_value_scales_many_rows():
    G.require_gpu()
    for e in (-126, -121, -114):
        b = R.Batch([70], [3000], 64, 1, 64, seed=1)
        b.v_scales[:] = 2.0 ** e
        b.v_pages[:] = b.v_pages.abs().clamp(min=64, max=127)
        b.k_scales[:] = 2.0 ** -10
        ATT._check(b, ATT._queries(70, 16, 64, BF16, 3))


def _odd_steps(x, dtype):
    """64-bit values to dtype, rounded once, wherever they lie."""
    m, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=-125) - 8)
    r = torch.round(x / step) * step
    return torch.where(r.abs() > torch.finfo(dtype).max, torch.sign(r) * float("inf"), r).to(torch.float32).to(dtype)


def test_rotated_queries_rounded_once():
    """bf16 queries up to the type's largest value and past it, next to the middle
    between two of them."""
    G.require_gpu()
    P, D, T = 16, 64, 512
    b = R.Batch([T], [0], P, 1, D, seed=1)
    g = torch.Generator().manual_seed(2)
    x = (torch.rand(T, 1, D, generator=g) * 0.3 + 0.85).mul(3.2e38).clamp(max=3.38e38).to(BF16)
    angle = torch.rand(b.width * P, D // 2, generator=g, dtype=F64) * 0.2
    cos, sin = angle.cos().float(), angle.sin().float()
    # cosines that put a value next to a middle: x c = (n + 1/2) step (1 + 2^-25 or so)
    mid = (torch.floor(x[:, 0, :D // 2].double() * 0.95 / 2.0 ** 120) + 0.5) * 2.0 ** 120
    cos[:T] = (mid / x[:, 0, :D // 2].double()).float()
    sin[:T] = 1e-8 * torch.randn(T, D // 2, generator=g)
    args = b.cuda()
    q_out = torch.empty(T, 1, D, dtype=BF16, device="cuda")
    mnb.append_kv_int8(x.cuda(), x.cuda(), cos.cuda(), sin.cuda(), *args, q=x.cuda(), q_out=q_out)
    torch.cuda.synchronize()
    want = torch.stack([R.rotate(x[t], cos[t], sin[t], False) for t in range(T)])
    assert torch.equal(q_out.cpu().view(torch.int16), _odd_steps(want, BF16).view(torch.int16))


@pytest.mark.parametrize("c,s", [(0.70710677, 0.70710677), (0.70710677, -0.70710677), (-1.0, 0.0), (0.6, 0.8), (8.0, 30.0), (-30.0, 20.0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_past_the_type(c, s, interleaved):
    """Rotated bf16 keys past fp32's range, of both signs, alone and in a page with
    small ones, before and after them; queries next to bf16's largest value."""
    G.require_gpu()
    P, D, T = 16, 64, 7
    big = torch.finfo(BF16).max
    for sizes in ((big, -big), (3e38, 3e38), (-3e38, 3e38), (2.9e38, 1e38), (1e38, -3.3e38), (-big, -big)):
        for place in (0, 3, 6):
            b = R.Batch([T], [5], P, 1, D, seed=place)
            b.k_scales[:] = 2.0 ** -4
            x = torch.zeros(T, 1, D)
            x[:] = torch.randn(T, 1, D, generator=torch.Generator().manual_seed(1))
            i, j = (8, 9) if interleaved else (4, 36)
            x[place, 0, i], x[place, 0, j] = sizes
            x = x.to(BF16)
            cos, sin = torch.full((b.width * P, D // 2), c), torch.full((b.width * P, D // 2), s)
            APP._run(b, x, x, x, cos, sin, interleaved)
            # and what comes after them, page by page
            b.starts, b.lengths, b.T = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([15], dtype=torch.int32), 3
            b.k_scales[b.k_scales == 0] = 2.0 ** -4
            y = torch.randn(3, 1, D).to(BF16)
            APP._run(b, y, y, y, cos, sin, interleaved)


def test_scales_up_to_the_largest():
    """Keys of 2^128 to 2^134: the scale is the largest power of two that fp32 has;
    from 2^134 on there is none, and it is NaN."""
    G.require_gpu()
    P, D = 16, 64
    for size in (2.0 ** 127, -2.0 ** 127, 3.3e38, -3.3e38):
        for by in (1.0, 2.0, 32.0, 64.0, 127.0, 128.0, 2.0 ** 60):
            b = R.Batch([2], [0], P, 1, D, seed=3)
            x = torch.zeros(2, 1, D)
            x[0, 0, 3], x[1, 0, 4] = size, 1.0
            x = x.to(BF16)
            cos, sin = torch.full((P, D // 2), by), torch.zeros(P, D // 2)
            args = b.cuda()
            mnb.append_kv_int8(x.cuda(), x.cuda(), cos.cuda(), sin.cuda(), *args)
            torch.cuda.synchronize()
            page = int(b.table[0, 0])
            y = float(x[0, 0, 3]) * by
            if -2.0 ** 134 <= y < 2.0 ** 134:
                R.append(b, x, x, cos, sin)
                for got, ref in zip(args[3:], b.cache()):
                    assert torch.equal(got.cpu(), ref)
            else:
                assert bool(torch.isnan(args[5][page, 0])) and bool((args[3][page, 0, :2] == 0).all())


def test_queries_without_a_usable_page():
    """A query that is not finite and sees no key: zeros, in every kernel."""
    G.require_gpu()
    for P in (16, 64):
        for new, hq in (([1, 2], 2), ([90, 1], 4), ([90, 1], 30)):
            b = R.Batch(new, [100] * len(new), P, 1, 64, seed=1)
            b.table[0] = -1
            q = ATT._queries(b.T, hq, 64, BF16, 1)
            clean = ATT._call(b, q)
            for bad in (float("nan"), float("inf")):
                q2 = q.clone()
                q2[0, 1, 3] = bad
                got = ATT._call(b, q2)
                assert bool((got[:new[0]] == 0).all())
                assert torch.equal(got, clean)
            # some usable pages only: the row is spoilt, and no other
            b.table[0, 1] = 0
            clean = ATT._call(b, q)
            got = ATT._call(b, q2)
            assert bool(torch.isnan(got[0, 1]).all())
            got[0, 1] = clean[0, 1]
            assert torch.equal(got, clean)


@pytest.mark.parametrize("P", [16, 32, 64, 256])
@pytest.mark.parametrize("new,hq", [([1, 2], 4), ([40], 16), ([70, 1], 64)], ids=["few", "shares", "tiles"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_that_are_no_powers_of_two(D, new, hq, P):
    G.require_gpu()
    b = R.Batch(new, [700, 333][:len(new)], P, 1, D, seed=P)
    g = torch.Generator().manual_seed(D)
    for i, scales in enumerate((b.k_scales, b.v_scales)):
        scales.mul_(torch.rand(scales.shape, generator=g) + 1)
        if i:
            scales[::3] *= 2.0 ** -12
    for dtype in (F16, BF16):
        ATT._check(b, ATT._queries(b.T, hq, D, dtype, 3))


def test_fractions_of_scales_are_exact_in_tiles():
    """One weight of 1 and one next to the middle between two fp16 values, a value
    scale likewise, integers whose products with it are: none but the weight may
    be rounded (two roundings more would pass the bound, all three up)."""
    G.require_gpu()
    P, D = 16, 64
    s = 1 + 0.51 * 2.0 ** -10
    half = lambda x: float(torch.tensor(x, dtype=F64).to(F16))
    n = [q for q in range(64, 128) if half((q + 0.5) * half(s)) > (q + 0.5) * half(s) * (1 + 2.0 ** -12.5)]
    assert half(s) > s and len(n) > 3
    b = R.Batch([5], [43], P, 1, D, seed=1)
    pages = b.table[0].tolist()
    b.k_pages[:] = 0
    b.k_scales[:] = 1
    b.v_scales[:] = s
    b.v_scales[pages[0]] = 1
    for p in pages[1:]:
        b.k_pages[p, :, :, 0] = -1
    b.k_pages[:, :, :, 1:] = 0
    for d in range(D):
        b.v_pages[pages[0], 0, d] = -n[d % len(n)] - 1      # -(n + 1/2): the sums are near zero
        for p in pages[1:]:
            b.v_pages[p, 0, d] = n[d % len(n)]
    q = torch.zeros(5, 64, D)
    q[:, :, 0] = 1
    ATT._check(b, q.to(F16), scale=-math.log(0.5 + 0.51 * 2.0 ** -11))


def test_max_tokens_past_any_length():
    """Bounds of the tokens up to the largest integer are bounds like others: the
    kernels of many rows."""
    G.require_gpu()
    b = R.Batch([300], [100], 32, 1, 64, seed=4)
    q = ATT._queries(b.T, 4, 64, BF16, 2)
    want = ATT._call(b, q, max_tokens=300)
    for most in (2 ** 31, 2 ** 62, 2 ** 63 - 1):
        c0 = mnb.mnb_counters_get()["launches"]
        got = ATT._call(b, q, max_tokens=most)
        assert mnb.mnb_counters_get()["launches"] - c0 == 3
        assert torch.equal(got, want)


def test_refusals_on_another_stream():
    """Wrong arguments are refused in the same manner where a stream is named."""
    G.require_gpu()
    b = R.Batch([3], [20], 16, 2, 64, seed=1)
    c = b.cuda()
    q = torch.zeros(3, 4, 64, dtype=F16, device="cuda")
    x, ids = torch.zeros(5, 64, dtype=F16, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    A, B = torch.zeros(2, 8, 64, dtype=F16, device="cuda"), torch.zeros(2, 30, 8, dtype=F16, device="cuda")
    y = torch.zeros(5, 30, dtype=F16, device="cuda")
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for error, call in ((ValueError, lambda: mnb.attention_int8(q[0], *c, q[0], stream=stream)),
                            (TypeError, lambda: mnb.attention_int8(q, c[0], 5, *c[2:], q, stream=stream)),
                            (TypeError, lambda: mnb.attention_int8(q, *c[:3], None, *c[4:], q, stream=stream)),
                            (ValueError, lambda: mnb.attention_int8(q, *c[:3], c[5], *c[4:], q, stream=stream)),
                            (ValueError, lambda: mnb.matmul_lora(x[0], ids, A, B, y, y, stream=stream)),
                            (ValueError, lambda: mnb.matmul_lora(x, ids, A[0, 0], B, y, y, stream=stream)),
                            (TypeError, lambda: mnb.matmul_lora(x, ids, A, None, y, y, stream=stream))):
            with pytest.raises(error):
                call()


def test_adapters_of_no_columns():
    """x of no columns, as torch lays it out (its rows one element apart): the base."""
    G.require_gpu()
    for m in (1, 2, 70):
        for n in (0, 3):
            x, A = torch.zeros(m, 0, dtype=F16, device="cuda"), torch.zeros(n, 8, 0, dtype=F16, device="cuda")
            B = torch.ones(n, 30, 8, dtype=F16, device="cuda")
            base = torch.randn(m, 30, device="cuda").to(F16)
            ids = torch.zeros(m, dtype=torch.int32, device="cuda")
            out = torch.empty_like(base)
            mnb.matmul_lora(x, ids, A, B, base, out)
            torch.cuda.synchronize()
            assert torch.equal(out, base)


@pytest.mark.parametrize("N,stride", [(4096, 4096), (4096, 4097), (4112, 4113), (4097, 4097), (4100, 4101)])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_base_at_the_ends_of_a_buffer(dtype, N, stride):
    """Adapters over a base that begins and ends within a word, next to other
    values: its first and last columns, and no value beside it."""
    G.require_gpu()
    m, K, rank, n = 600, 96, 16, 3
    g = torch.Generator().manual_seed(N + stride)
    x = torch.randn(m, K, generator=g).to(dtype)
    ids = torch.randint(-1, n, (m,), generator=g).to(torch.int32)
    A = (torch.randn(n, rank, K, generator=g) * 0.1).to(dtype)
    B = torch.randn(n, N, rank, generator=g).to(dtype)
    for at in (0, 1, 3):
        for in_place in (False, True):
            size = (m - 1) * stride + N
            around = torch.full((at + size + 2,), float("nan"), dtype=dtype)
            values = torch.randn(size, generator=g).to(dtype)
            around[at:at + size] = values
            dev = around.cuda()
            base = torch.as_strided(dev, (m, N), (stride, 1), at)
            room = dev if in_place else torch.full_like(dev, 5.0)
            out = torch.as_strided(room, (m, N), (stride, 1), at)
            want = base.clone()
            plain = torch.empty(m, N, dtype=dtype, device="cuda")
            mnb.matmul_lora(x.cuda(), ids.cuda(), A.cuda(), B.cuda(), want, plain)
            before = room.clone()
            mnb.matmul_lora(x.cuda(), ids.cuda(), A.cuda(), B.cuda(), base, out)
            torch.cuda.synchronize()
            assert torch.equal(out, plain)
            inside = torch.zeros_like(room, dtype=torch.bool)
            torch.as_strided(inside, (m, N), (stride, 1), at).fill_(True)
            assert torch.equal(room[~inside].view(torch.int16), before[~inside].view(torch.int16))
            if not in_place:
                assert torch.equal(dev.cpu().view(torch.int16), around.view(torch.int16))
