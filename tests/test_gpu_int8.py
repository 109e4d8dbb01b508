"""quantize_rows_int8 and matmul_int8 on the GPU against exact arithmetic on
the CPU.

Quantised rows and scales have to be equal: the integers are the rounding of
an exact quotient, the scale one correctly rounded division.

Products: the integer sum S is exact.  The call rounds S to fp32, multiplies
by the two scales and adds the bias in fp32 (four roundings of at most 2^-24,
relative to the product or to the sum), and rounds once to fp16 or bf16 (half
a step: eps/2 of the value, or 2^-25 below fp16's smallest normal number).
So with P = S a b and y = P + bias in exact arithmetic
    |out - y| <= (eps / 2) |y| (1 + 2^-10) + 4 * 2^-24 (|P| + |y|) + 2^-25,
and where S stays below 2^24 and both scales are powers of two the result is
the rounding of the exact value, bit for bit.
"""
import numpy as np
import pytest
import torch

import block_wise_int4_matmulnbits_amd as mnb
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _rows(m, K, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, K, generator=g) * scale
    return (x * (torch.rand(m, 1, generator=g) * 4 + 0.1)).to(dtype)


def _quantize_ref(x):
    """(int8 rows, fp32 scales), numpy in 64 bits."""
    v = x.to(torch.float64).numpy()
    finite = np.isfinite(v).all(axis=1)
    top = np.abs(np.where(np.isfinite(v), v, 0)).max(axis=1) if v.shape[1] else np.zeros(len(v))
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where((top > 0)[:, None], np.rint(127.0 * v / top[:, None]), 0.0)
        q = np.where(finite[:, None], q, 0.0)
        s = np.where(finite, top.astype(np.float32) / np.float32(127), np.float32("nan"))
    return q.astype(np.int8), s.astype(np.float32)


def _gpu_quantize(x, stream=None):
    m, K = x.shape
    q = torch.full((m + 2, max(K, 1)), 85, dtype=torch.int8, device="cuda")
    s = torch.full((m + 2,), 7.0, device="cuda")
    qq = q.view(-1)[:m * K].view(m, K)
    mnb.quantize_rows_int8(x.cuda(), qq, s[:m], stream=stream)
    torch.cuda.synchronize()
    assert (q.view(-1)[m * K:] == 85).all() and (s[m:] == 7.0).all()   # what lies behind the rows is left alone
    return qq.cpu().numpy(), s[:m].cpu().numpy()


def _check_quantize(x):
    q, s = _gpu_quantize(x)
    rq, rs = _quantize_ref(x)
    assert np.array_equal(q, rq), "%d integers differ" % int((q != rq).sum())
    assert np.array_equal(s, rs, equal_nan=True)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,K", [(1, 16), (1, 4096), (3, 48), (7, 1040), (2, 16400), (5, 14336), (300, 272),
                                 (2, 70000), (1, 131056), (4100, 64), (33, 8208), (1, 0),
                                 (1100, 2064), (1031, 4112), (1025, 8400), (1024, 16400)])
def test_quantize(m, K, dtype):
    G.require_gpu()
    _check_quantize(_rows(m, K, dtype, 7 * m + K))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_quantize_ties_and_extremes(dtype):
    """Every pair (max, value) of a small grid: exact ties (value = max
    (2n+1)/254), neighbours of them, subnormal and largest maxima, rows of
    zeros, and infinities and NaN."""
    G.require_gpu()
    rows = []
    for top in (127.0, 254.0, 1.0, 2.0, 63.5, 0.4375, 1.9921875, 96.0, 3.0, torch.finfo(dtype).max,
                torch.finfo(dtype).tiny, torch.finfo(dtype).smallest_normal * 0.25):
        n = torch.arange(-127, 128, dtype=torch.float64)
        v = torch.cat((n * top / 127, (n + 0.5) * top / 127)).clamp(-top, top).to(dtype).to(torch.float64)
        v = torch.cat((v, torch.tensor([top, -top], dtype=torch.float64)))
        rows.append(torch.nn.functional.pad(v, (0, 528 - v.numel())).to(dtype))
    x = torch.stack(rows)
    zero = torch.zeros(1, 528, dtype=dtype)
    zero[0, 3] = -0.0
    bad = [x[0:1].clone() for _ in range(4)]
    for b, value, at in zip(bad, (float("inf"), -float("inf"), float("nan"), -float("nan")), (0, 527, 100, 511)):
        b[0, at] = value
    _check_quantize(torch.cat([x, zero] + bad))


def _product(x, a_scales, W, b_scales, bias, out_dtype, stream=None, workspace=None):
    m, N = x.shape[0], W.shape[0]
    out = torch.full((m * N + 16,), -1, dtype=torch.int16, device="cuda")
    mnb.matmul_int8(x, a_scales, W, b_scales, bias, out[:m * N].view(out_dtype).view(m, N), workspace=workspace,
                    stream=stream)
    torch.cuda.synchronize()
    assert (out[m * N:] == -1).all()
    return out[:m * N].view(out_dtype).view(m, N).cpu()


def _inputs(m, K, N, seed, full=False):
    g = torch.Generator().manual_seed(seed)
    lo = -128 if full else -127
    A = torch.randint(lo, 128, (m, K), generator=g, dtype=torch.int8)
    W = torch.randint(lo, 128, (N, K), generator=g, dtype=torch.int8)
    a = torch.rand(m, generator=g) * 0.02 + 1e-3
    b = torch.rand(N, generator=g) * 1e-3 + 1e-5
    bias = torch.randn(N, generator=g) * 3
    return A, a, W, b, bias


def _check(out, A, a, W, b, bias, out_dtype):
    S = torch.matmul(A.double(), W.double().t())
    P = S * a.double()[:, None] * b.double()[None, :]
    y = P if bias is None else P + bias.double()[None, :]
    tol = torch.finfo(out_dtype).eps / 2 * y.abs() * (1 + 2.0 ** -10) + 4 * 2.0 ** -24 * (P.abs() + y.abs()) + 2.0 ** -25
    err = (out.double() - y).abs()
    assert bool((err <= tol).all()), "worst %g of its tolerance" % float((err / tol).max())


SHAPES = [(1, 16, 1), (1, 4096, 64), (2, 48, 17), (3, 64, 33), (5, 1040, 100), (8, 14336, 70), (16, 80, 16),
          (17, 128, 40), (31, 4112, 65), (33, 272, 129), (64, 512, 64), (65, 2064, 200), (100, 1024, 131),
          (129, 96, 257), (255, 144, 300), (256, 256, 256), (300, 640, 520), (513, 112, 70), (1000, 400, 600),
          (4, 32768, 48), (40, 20480, 30), (4, 131056, 5), (200, 0, 9), (1, 0, 5)]


@pytest.mark.parametrize("m,K,N", SHAPES)
def test_product_of_integers(m, K, N):
    G.require_gpu()
    A, a, W, b, bias = _inputs(m, K, N, 3 * m + K + N)
    dev = [t.cuda() for t in (A, a, W, b, bias)]
    for out_dtype, use_bias in ((F16, False), (BF16, True)):
        out = _product(*dev[:4], dev[4] if use_bias else None, out_dtype)
        _check(out, A, a, W, b, bias if use_bias else None, out_dtype)


@pytest.mark.parametrize("m,K,N", [(300, 48, 50000), (1025, 144, 9001), (700, 272, 9001), (200, 400, 9000),
                                   (250, 1040, 7003), (1000, 400, 600), (60, 2064, 8003), (255, 144, 300)])
def test_every_tile_and_the_rows_kernel_give_the_same_bits(m, K, N):
    """Shapes that the choice by cost gives each of the seven tiles, with ragged
    edges, and the first rows of each alone (the kernel for few rows)."""
    G.require_gpu()
    A, a, W, b, bias = _inputs(m, K, N, m + K + N, full=True)
    dev = [t.cuda() for t in (A, a, W, b, bias)]
    for out_dtype in (F16, BF16):
        out = _product(*dev, out_dtype)
        _check(out, A, a, W, b, bias, out_dtype)
        few = _product(dev[0][:5].contiguous(), dev[1][:5].contiguous(), *dev[2:], out_dtype)
        assert torch.equal(few.view(torch.int16), out[:5].view(torch.int16))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,K,N", SHAPES)
def test_product_of_activations(m, K, N, dtype):
    """fp16 and bf16 rows: the bits of quantize_rows_int8 followed by the
    integer product."""
    G.require_gpu()
    x = _rows(m, K, dtype, m + K + N)
    _, _, W, b, bias = _inputs(m, K, N, 5 * m + K + N)
    x, W, b, bias = x.cuda(), W.cuda(), b.cuda(), bias.cuda()
    q = torch.empty(m, K, dtype=torch.int8, device="cuda")
    s = torch.empty(m, device="cuda")
    mnb.quantize_rows_int8(x, q, s)
    rq, rs = _quantize_ref(x.cpu())
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    for out_dtype in (F16, BF16):
        got = _product(x, None, W, b, bias, out_dtype)
        assert torch.equal(got.view(torch.int16), _product(q, s, W, b, bias, out_dtype).view(torch.int16))
        _check(got, q.cpu(), s.cpu(), W.cpu(), b.cpu(), bias.cpu(), out_dtype)


@pytest.mark.parametrize("m,N", [(1, 40), (9, 40), (40, 200), (300, 300)])
def test_sums_are_exact(m, N):
    """Unit scales and integers whose sums stay below 2^11: the fp16 output is
    the sum itself, so one product lost or counted twice shows."""
    G.require_gpu()
    g = torch.Generator().manual_seed(m)
    K = 1584
    A = torch.randint(-1, 2, (m, K), generator=g, dtype=torch.int8)
    W = torch.randint(-1, 2, (N, K), generator=g, dtype=torch.int8)
    one = torch.ones(max(m, N))
    out = _product(A.cuda(), one[:m].cuda(), W.cuda(), one[:N].cuda(), None, F16)
    S = torch.matmul(A.double(), W.double().t())
    assert float(S.abs().max()) < 2048
    assert torch.equal(out.double(), S)


@pytest.mark.parametrize("m", [1, 20, 200])
def test_largest_sums(m):
    """-128 * -128 over the longest K: 2147221504, the largest sum there is;
    and its negative neighbour -128 * 127."""
    G.require_gpu()
    K, N = mnb.MNB_MAX_K_INT8, 40
    A = torch.full((m, K), -128, dtype=torch.int8, device="cuda")
    W = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    W[1::2] = 127
    s = torch.full((max(m, N),), 2.0 ** -16, device="cuda")
    out = _product(A, s[:m], W, s[:N], None, BF16)
    want = torch.tensor([128.0 * 128 * K, -128.0 * 127 * K], dtype=torch.float64) * 2.0 ** -32
    assert torch.equal(out, want.to(BF16).repeat(m, N // 2))


@pytest.mark.parametrize("m", [2, 24, 150])
def test_rows_without_finite_scale_and_zero_rows(m):
    """A row with a NaN or an infinity gives a row of NaN and leaves the others
    alone; a row of zeros gives the bias; a product past fp16 gives infinity."""
    G.require_gpu()
    K, N = 96, 50
    x = _rows(m, K, F16, 11)
    x[0, 5] = float("inf")
    x[1] = 0
    _, _, W, b, bias = _inputs(m, K, N, 12)
    out = _product(x.cuda(), None, W.cuda(), b.cuda(), bias.cuda(), F16)
    assert out[0].isnan().all()
    assert torch.equal(out[1], bias.to(F16))
    assert out[2:].isfinite().all()
    big = _product(x.cuda(), None, W.cuda(), (b * 0 + 3e4).cuda(), None, F16)
    assert out[2:].numel() == 0 or big[2:].isinf().any()


@pytest.mark.parametrize("m,a", [(1, "i8"), (8, "f16"), (20, "i8"), (300, "i8")])
def test_offsets_past_32_bits(m, a):
    """Weights of more than 2^32 bytes: columns from all along them against the
    CPU."""
    G.require_gpu()
    K, N = 16384, 270001                     # 4.42e9 bytes
    g = torch.Generator(device="cuda").manual_seed(5)
    W = torch.empty(N, K, dtype=torch.int8, device="cuda")
    for n in range(0, N, 65536):
        W[n:n + 65536] = torch.randint(-127, 128, W[n:n + 65536].shape, generator=g, device="cuda", dtype=torch.int8)
    A, sa, _, _, _ = _inputs(m, K, 1, 3)
    b = torch.rand(N, generator=g, device="cuda") * 1e-3
    if a == "i8":
        out = _product(A.cuda(), sa.cuda(), W, b, None, BF16)
        q, s = A, sa
    else:
        x = _rows(m, K, F16, 4)
        out = _product(x.cuda(), None, W, b, None, BF16)
        q, s = (torch.from_numpy(t) for t in _quantize_ref(x))
    for cols in (slice(0, 16), slice(131060, 131090), slice(262130, 262160), slice(N - 33, N)):
        _check(out[:, cols], q, s, W[cols].cpu(), b[cols].cpu(), None, BF16)


def test_streams_and_graph():
    """A call on another stream, two streams at once, and captured calls (each
    with its own workspace) replayed with other inputs between eager calls."""
    G.require_gpu()
    K, N = 2048, 1024
    _, _, W, b, bias = (t.cuda() for t in _inputs(1, K, N, 1))
    for m in (4, 70):
        xs = [_rows(m, K, BF16, 20 + i).cuda() for i in range(4)]
        want = [_product(x, None, W, b, bias, F16) for x in xs]
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [torch.empty(m, N, dtype=F16, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        for i in range(4):
            mnb.matmul_int8(xs[i], None, W, b, bias, outs[i], stream=streams[i % 2])
        torch.cuda.synchronize()
        for i in range(4):
            assert torch.equal(outs[i].cpu(), want[i])
        x_in = xs[0].clone()
        outs2 = [torch.empty(m, N, dtype=F16, device="cuda") for _ in range(2)]
        graphs = []
        for o in outs2:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                mnb.matmul_int8(x_in, None, W, b, bias, o)
            graphs.append(g)
        for i in range(4):
            x_in.copy_(xs[i])
            torch.cuda.synchronize()
            for o, g, s in zip(outs2, graphs, streams):
                o.fill_(-1)
            torch.cuda.synchronize()
            for g, s in zip(graphs, streams):      # both replays in flight at once
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            eager = _product(xs[(i + 1) % 4], None, W, b, bias, F16)
            assert torch.equal(eager, want[(i + 1) % 4])
            for o in outs2:
                assert torch.equal(o.cpu(), want[i])


def test_workspace_of_the_caller_and_counters():
    """A dirty workspace of exactly the stated size; what lies behind it stays."""
    G.require_gpu()
    m, K, N = 200, 512, 300
    x = _rows(m, K, F16, 3).cuda()
    _, _, W, b, _ = (t.cuda() for t in _inputs(1, K, N, 2))
    need = mnb.mnb_int8_workspace(mnb.MNB_F16, m, K, N)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    c0 = mnb.mnb_counters_get()
    got = _product(x, None, W, b, None, BF16, workspace=ws[:need])
    c1 = mnb.mnb_counters_get()
    assert c1["calls"] == c0["calls"] + 1 and c1["launches"] - c0["launches"] in (1, 2)
    assert (ws[need:] == 255).all()
    assert torch.equal(got, _product(x, None, W, b, None, BF16))
    with pytest.raises(mnb.MnbError):
        mnb.matmul_int8(x, None, W, b, None, torch.empty(m, N, dtype=F16, device="cuda"), workspace=ws[:need - 1])


def test_binding_refusals():
    G.require_gpu()
    A, a, W, b, bias = (t.cuda() for t in _inputs(4, 64, 8, 1))
    out = torch.empty(4, 8, dtype=F16, device="cuda")
    for args in ((A, None, W, b, None, out), (A, a[:3], W, b, None, out), (A, a, W[:, :48], b, None, out),
                 (A, a, W, b[:7], None, out), (A, a, W, b, bias[:7], out), (A, a, W, b, None, out[:3]),
                 (A.half(), a, W, b, None, out), (A[:, ::2], a, W[:, :32].contiguous(), b, None, out),
                 (A, a, W.cpu(), b, None, out)):
        with pytest.raises(ValueError):
            mnb.matmul_int8(*args)
    for args in ((A.float(), None, W, b, None, out), (A, a.half(), W, b, None, out), (A, a, W.half(), b, None, out),
                 (A, a, W, b, None, out.float())):
        with pytest.raises(TypeError):
            mnb.matmul_int8(*args)
