"""matmul_lora against its formula in 64 bits."""
import pytest
import torch

import block_wise_int4_matmulnbits_amd as mnb
from tests import gpu_util as G
from tests import kv_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _make(m, K, N, rank, n, dtype, out, seed, run=1, none=0.2):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, K, generator=g).to(dtype)
    A = (torch.randn(n, rank, K, generator=g) * max(K, 1) ** -0.5).to(dtype)
    B = torch.randn(n, N, rank, generator=g).to(dtype)
    ids = torch.randint(0, max(n, 1), (m // run + 1,), generator=g).repeat_interleave(run)[:m].to(torch.int32)
    off = torch.rand(m, generator=g) < none
    ids[off] = torch.tensor([-1, n, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 4, (int(off.sum()),), generator=g)].to(torch.int32)
    scaling = torch.rand(n, generator=g) * 4 - 2
    base = (torch.randn(m, N, generator=g) * 3).to(out)
    return x, ids, A, B, scaling, base


def _check(x, ids, A, B, scaling, base, out_dtype, in_place=False):
    dev = [None if t is None else t.cuda() for t in (x, ids, A, B, base)]
    out = dev[4] if in_place else torch.full((x.shape[0], B.shape[1]), 9.0, dtype=out_dtype, device="cuda")
    got = mnb.matmul_lora(*dev, out, scaling=None if scaling is None else scaling.cuda())
    torch.cuda.synchronize()
    assert got is out
    want, tol = R.lora(x, ids, A, B, scaling, base)
    R.check_rows(out.cpu(), want, tol, out_dtype)
    return out.cpu()


SHAPES = [
    # m, K, N, rank, adapters, run
    (1, 16, 1, 8, 1, 1), (1, 4096, 4096, 16, 8, 1), (2, 256, 65, 8, 3, 1), (7, 1040, 129, 24, 5, 1),
    (16, 512, 256, 64, 16, 1), (17, 528, 300, 32, 40, 1), (64, 1024, 1000, 64, 32, 1), (65, 272, 257, 16, 3, 9),
    (100, 2064, 511, 40, 6, 1), (300, 144, 64, 128, 7, 50), (129, 512, 320, 200, 4, 20), (70, 96, 33, 256, 2, 1),
    (1000, 32, 16, 8, 5, 333), (64, 64, 25001, 40, 20, 1), (1100, 160, 40, 8, 3, 100), (1030, 160, 33, 32, 3, 1),
    (1024, 144, 17, 48, 2, 7), (1025, 96, 20, 128, 2, 300),
]


@pytest.mark.parametrize("dtype,out", [(F16, F16), (BF16, BF16), (BF16, F16), (F16, BF16)],
                         ids=["f16", "bf16", "bf16_f16", "f16_bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_rows(shape, dtype, out):
    G.require_gpu()
    m, K, N, rank, n, run = shape
    x, ids, A, B, scaling, base = _make(m, K, N, rank, n, dtype, out, m + K, run)
    got = _check(x, ids, A, B, scaling, base, out)
    none = (ids < 0) | (ids >= n)
    assert torch.equal(got[none], base[none])


def test_forms():
    """No base, no scaling, in place, no adapters at all, K of 0."""
    G.require_gpu()
    for dtype in (F16, BF16):
        x, ids, A, B, scaling, base = _make(37, 320, 203, 16, 4, dtype, dtype, 5)
        got = _check(x, ids, A, B, None, None, dtype)
        assert bool((got[(ids < 0) | (ids >= 4)] == 0).all())
        _check(x, ids, A, B, scaling, base, dtype, in_place=True)
        got = _check(x, ids, A[:0], B[:0], scaling[:0], base, dtype)
        assert torch.equal(got, base)
        got = _check(x[:, :0], ids, A[:, :, :0], B, scaling, base, dtype)
        assert torch.equal(got, base)


def test_range_of_fp16():
    """Sums past fp16's range and far below it between the two products."""
    G.require_gpu()
    for size in (1e-6, 1e-3, 300.0):
        x, ids, A, B, scaling, base = _make(20, 256, 100, 16, 3, F16, BF16, 2)
        x = (x.float() * size).to(F16)
        A = (A.float() * 64).to(F16)
        _check(x, ids, A, B, scaling, base, BF16)


def test_not_finite_stays_in_its_row():
    G.require_gpu()
    for dtype in (F16, BF16):
        x, ids, A, B, scaling, base = _make(40, 128, 70, 8, 3, dtype, dtype, 4, none=0.0)
        clean = _check(x, ids, A, B, scaling, base, dtype)
        for bad in (float("nan"), float("inf")):
            x2 = x.clone()
            x2[11, 5] = bad
            out = torch.empty_like(base).cuda()
            mnb.matmul_lora(x2.cuda(), ids.cuda(), A.cuda(), B.cuda(), base.cuda(), out, scaling=scaling.cuda())
            out = out.cpu()
            assert not bool(torch.isfinite(out[11]).any())
            out[11] = clean[11]
            assert torch.equal(out, clean)


def test_adapters_do_not_mix():
    """A row's bits do not depend on the other rows' adapters, nor on weights of
    adapters that no row uses."""
    G.require_gpu()
    x, ids, A, B, scaling, base = _make(64, 512, 256, 16, 8, BF16, BF16, 6, none=0.0)
    want = _check(x, ids, A, B, scaling, base, BF16)
    for a in range(8):
        only = torch.where(ids == a, ids, torch.full_like(ids, -1))
        A2, B2 = torch.full_like(A, float("nan")), torch.full_like(B, float("nan"))
        A2[a], B2[a] = A[a], B[a]
        got = _call(x, only, A2, B2, scaling, base)
        assert torch.equal(got[ids == a], want[ids == a]) and torch.equal(got[ids != a], base[ids != a])


def _call(x, ids, A, B, scaling, base):
    out = torch.empty_like(base).cuda()
    mnb.matmul_lora(x.cuda(), ids.cuda(), A.cuda(), B.cuda(), base.cuda(), out, scaling=scaling.cuda())
    torch.cuda.synchronize()
    return out.cpu()


def test_strides_and_streams():
    """Slices of wider buffers at odd columns; a raw stream handle; a workspace."""
    G.require_gpu()
    for m in (5, 200):
        x, ids, A, B, scaling, base = _make(m, 256, 101, 16, 4, F16, F16, 7)
        want = _call(x, ids, A, B, scaling, base)
        xs = torch.zeros(m, 300 + 20, dtype=F16, device="cuda")
        xs[:, 8:264] = x.cuda()
        wide = torch.full((m, 333), 4.0, dtype=F16, device="cuda")
        wide[:, 13:114] = base.cuda()
        dev = [t.cuda() for t in (ids, A, B)]
        ws = torch.empty(mnb.mnb_lora_workspace(m, 256, 101, 16, 4), dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        s = scaling.cuda()
        torch.cuda.synchronize()
        mnb.matmul_lora(xs[:, 8:264], *dev, wide[:, 13:114], wide[:, 201:302], scaling=s, workspace=ws, stream=side.cuda_stream)
        mnb.matmul_lora(xs[:, 8:264], *dev, wide[:, 13:114], wide[:, 13:114], scaling=s, workspace=ws, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(wide[:, 201:302].cpu(), want) and torch.equal(wide[:, 13:114].cpu(), want)
        wide[:, 201:302] = 4.0
        wide[:, 13:114] = 4.0
        assert bool((wide == 4.0).all())


def test_captured():
    G.require_gpu()
    sets = [_make(24, 512, 300, 16, 5, BF16, BF16, i) for i in range(3)]
    dev = [t.cuda() for t in sets[0]]
    x, ids, A, B, scaling, base = dev
    out = torch.empty_like(base)
    mnb.matmul_lora(x, ids, A, B, base, out, scaling=scaling)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mnb.matmul_lora(x, ids, A, B, base, out, scaling=scaling)
    for i in (1, 2, 0, 2):
        for dst, src in zip(dev, sets[i]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), _call(*sets[i]))


WIDE = [
    # m, K, N, rank, adapters, run: enough columns and rows for the wide second launch
    (300, 48, 27136, 16, 9, 40), (300, 48, 27137, 16, 9, 7), (9, 32, 130571, 8, 3, 1), (70, 32, 65539, 136, 3, 30),
    (40, 96, 131073, 72, 2, 5), (4099, 16, 2049, 24, 5, 600),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", WIDE, ids=["x".join(map(str, s)) for s in WIDE])
def test_wide(shape, dtype):
    G.require_gpu()
    m, K, N, rank, n, run = shape
    x, ids, A, B, scaling, base = _make(m, K, N, rank, n, dtype, dtype, m + N, run)
    dev = [t.cuda() for t in (x, ids, A, B, base)]
    out = torch.full((m, N), 9.0, dtype=dtype, device="cuda")
    mnb.matmul_lora(*dev, out, scaling=scaling.cuda())
    torch.cuda.synchronize()
    none = (ids < 0) | (ids >= n)
    out = out.cpu()
    assert torch.equal(out[none], base[none])
    some = torch.arange(0, m, max(1, m // 40))          # rows against 64 bits
    want, tol = R.lora(x[some], ids[some], A, B, scaling, base[some])
    R.check_rows(out[some], want, tol, dtype)
    # the other rows: the same values as alone
    got = torch.empty(m, N, dtype=dtype, device="cuda")
    mnb.matmul_lora(*dev[:4], None, got, scaling=scaling.cuda())
    torch.cuda.synchronize()
    got = got.cpu()
    assert bool((got[none] == 0).all())
    want, tol = R.lora(x[some], ids[some], A, B, scaling, None)
    R.check_rows(got[some], want, tol, dtype)
    size = 2.0 ** -6 * (got.float().abs() + base.float().abs() + 1)
    assert bool(((out.float() - base.float() - got.float()).abs() <= size).all())


def test_adapters_that_are_not_finite():
    """An adapter whose weights or scaling are not finite spoils its own rows alone."""
    G.require_gpu()
    for m, N, dtype in ((12, 130, F16), (70, 130, BF16), (300, 27137, BF16)):
        x, ids, A, B, scaling, base = _make(m, 64, N, 24, 5, dtype, dtype, 8, none=0.1)
        clean = _call(x, ids, A, B, scaling, base)
        for bad in (float("nan"), float("inf")):
            for which in range(3):
                w = [A.clone(), B.clone(), scaling.clone()]
                w[which][2] = bad
                got = _call(x, ids, *w, base)
                assert torch.equal(got[ids != 2], clean[ids != 2])
                assert not bool(torch.isfinite(got[ids == 2]).any())


def test_two_graphs_of_one_workspace():
    G.require_gpu()
    sets = [_make(m, 512, 300, 16, 5, BF16, BF16, m) for m in (24, 130)]
    ws = torch.empty(max(mnb.mnb_lora_workspace(m, 512, 300, 16, 5) for m in (24, 130)), dtype=torch.uint8, device="cuda")
    work = []
    for s in sets:
        x, ids, A, B, scaling, base = [t.cuda() for t in s]
        out = torch.empty_like(base)
        mnb.matmul_lora(x, ids, A, B, base, out, scaling=scaling, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mnb.matmul_lora(x, ids, A, B, base, out, scaling=scaling, workspace=ws)
        work.append((graph, (x, ids, A, B, scaling, base), out, _call(*s)))
    for i in (0, 1, 1, 0, 1, 0):
        graph, _, out, want = work[i]
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)
        _call(*sets[1 - i])


def test_wide_within_a_buffer():
    """The wide second launch on rows at odd columns of a wider buffer, in place and
    not: the columns around them keep their bits."""
    G.require_gpu()
    m, K, N, rank = 300, 48, 27137, 16
    for dtype, at, wide in ((F16, 3, 27150), (BF16, 8, 27145), (F16, 1, 27140)):
        x, ids, A, B, scaling, base = _make(m, K, N, rank, 5, dtype, dtype, 9, 30)
        want = _call(x, ids, A, B, scaling, base)
        buf = torch.full((m, wide), 4.0, dtype=dtype, device="cuda")
        buf[:, at:at + N] = base.cuda()
        dev = [t.cuda() for t in (x, ids, A, B)]
        other = torch.full((m, wide + 1), 4.0, dtype=dtype, device="cuda")
        mnb.matmul_lora(*dev, buf[:, at:at + N], other[:, at:at + N], scaling=scaling.cuda())
        mnb.matmul_lora(*dev, buf[:, at:at + N], buf[:, at:at + N], scaling=scaling.cuda())
        torch.cuda.synchronize()
        for t in (buf, other):
            assert torch.equal(t[:, at:at + N].cpu(), want)
            t[:, at:at + N] = 4.0
            assert bool((t == 4.0).all())
