"""attention_int8 against its formula in 64 bits."""
import pytest
import torch

import block_wise_int4_matmulnbits_amd as mnb
from tests import gpu_util as G
from tests import kv_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _queries(T, hq, D, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hq, D, generator=g)
    channels = torch.rand(hq, D, generator=g)
    return (x * torch.where(channels > 0.97, 8.0, 1.0) * size).to(dtype)


def _call(b, q, scale=None, out=None, **kw):
    args = b.cuda()
    if out is None:
        out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    got = mnb.attention_int8(q.cuda(), *args, out, scale=scale, **kw)
    torch.cuda.synchronize()
    assert got is out
    return out.cpu()


def _check(b, q, scale=None, **kw):
    got = _call(b, q, scale, **kw)
    want, tol = R.attention(b, q, q.shape[2] ** -0.5 if scale is None else scale)
    used = int(b.starts[-1])
    R.check_rows(got[:used], want[:used], tol[:used], q.dtype)
    assert bool((got[used:] == 9.0).all())
    return got


SHAPES = [
    # new, before, P, query heads, heads, D
    ([1], [0], 16, 1, 1, 64),
    ([1], [62], 64, 4, 1, 128),
    ([1], [63], 64, 8, 2, 128),
    ([1], [64], 64, 8, 2, 128),
    ([1], [2048], 64, 8, 2, 128),
    ([1], [1500], 16, 5, 1, 256),
    ([1, 1, 1, 1, 1, 1], [0, 1, 15, 16, 200, 999], 16, 6, 3, 64),
    ([1, 0, 1, 0], [40, 40, 0, 0], 32, 2, 2, 128),
    ([3, 1, 5, 0, 2], [0, 700, 61, 13, 126], 32, 8, 2, 128),
    ([7], [250], 128, 16, 1, 64),
    ([2, 9], [10, 300], 256, 24, 2, 128),
    ([40, 1, 17], [0, 100, 33], 64, 4, 2, 128),
    ([130], [70], 16, 3, 3, 64),
    ([33, 65], [500, 0], 32, 8, 1, 256),
    ([300], [0], 64, 4, 1, 128),
    # many rows: tiles, with and without their keys split over workgroups
    ([65], [0], 64, 1, 1, 128),
    ([1, 200, 3, 90], [500, 0, 70, 1000], 32, 8, 2, 128),
    ([257, 70], [3, 64], 16, 2, 2, 128),
    ([120, 0, 121], [0, 9, 700], 16, 2, 1, 256),
    ([600], [130], 128, 64, 16, 64),
    ([1100], [0], 64, 60, 30, 128),
    ([9], [4000], 64, 64, 1, 128),
    ([90, 333], [2000, 1], 256, 5, 5, 64),
    ([65], [0], 64, 36, 1, 128),
    ([1, 200, 3, 90], [500, 0, 70, 1000], 32, 16, 2, 128),
    ([257, 70], [3, 64], 16, 8, 2, 128),
    ([66, 65], [4000, 100], 16, 16, 4, 128),
    ([130, 300], [33, 0], 64, 6, 1, 256),
    ([9, 9, 9, 9], [5000, 1, 0, 640], 16, 64, 1, 64),
    ([33], [9000], 32, 64, 1, 128),
    ([130, 4], [700, 90], 64, 16, 16, 64),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_rows(shape, dtype):
    G.require_gpu()
    new, before, P, hq, heads, D = shape
    b = R.Batch(new, before, P, heads, D, seed=P + D + len(new), extra=3)
    _check(b, _queries(b.T, hq, D, dtype, 7 * P + hq), max_tokens=max(new))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long(D):
    """A length that many workgroups share, joined in the order of the keys."""
    G.require_gpu()
    b = R.Batch([1, 2], [33333, 4099], 64, 1, D, seed=D)
    _check(b, _queries(b.T, 4, D, BF16, D))


def test_large_scores():
    """Weights that all but one key lose, and the scale's sign."""
    G.require_gpu()
    for scale in (2.0, -0.5, 0.0, 1e-3):
        for dtype in (F16, BF16):
            b = R.Batch([2, 1], [90, 700], 16, 2, 64, seed=5)
            b.k_scales = torch.full_like(b.k_scales, 2.0 ** -4)
            _check(b, _queries(b.T, 4, 64, dtype, 3), scale=scale)


def test_scales_far_apart():
    """Pages whose scales differ by up to 2^60, pages of zeros, zero queries."""
    G.require_gpu()
    for P in (16, 64):
        b = R.Batch([1, 2], [190, 333], P, 2, 128, seed=8)
        g = torch.Generator().manual_seed(1)
        b.v_scales = torch.exp2(torch.randint(-40, 20, b.v_scales.shape, generator=g).float())
        b.k_scales = torch.exp2(torch.randint(-30, -5, b.k_scales.shape, generator=g).float())
        b.v_scales[int(b.table[0, 0])] = 0
        b.k_scales[int(b.table[1, 1])] = 0
        q = _queries(b.T, 4, 128, BF16, 4)
        q[1] = 0
        _check(b, q)
        b.v_scales[:] = 0
        got = _call(b, q)
        assert bool((got == 0).all())


def test_scales_far_apart_many_rows():
    """The same for tiles: value scales that differ within a unit and from page to
    page, pages of zeros, rows that see only some of them."""
    G.require_gpu()
    for P in (16, 32, 64):
        for D in (64, 128):
            b = R.Batch([150], [40], P, 1, D, seed=8)
            g = torch.Generator().manual_seed(P)
            b.v_scales = torch.exp2(torch.randint(-20, 10, b.v_scales.shape, generator=g).float())
            b.k_scales = torch.exp2(torch.randint(-30, -5, b.k_scales.shape, generator=g).float())
            b.v_scales[int(b.table[0, 0])] = 0
            b.k_scales[int(b.table[0, 1])] = 0
            q = _queries(b.T, 3, D, BF16, 4)
            q[1] = 0
            _check(b, q)
            b.v_scales[:] = 0
            assert bool((_call(b, q) == 0).all())


@pytest.mark.parametrize("hq", [4, 30])
def test_large_scores_many_rows(hq):
    G.require_gpu()
    for scale in (2.0, -0.5, 0.0, 1e-3):
        for dtype in (F16, BF16):
            b = R.Batch([100, 70], [90, 300], 16, 2, 64, seed=5)
            b.k_scales = torch.full_like(b.k_scales, 2.0 ** -4)
            _check(b, _queries(b.T, hq, 64, dtype, 3), scale=scale)


@pytest.mark.parametrize("hq", [2, 24])
def test_not_finite_many_rows(hq):
    """Rows of tiles that do not see a page whose scale is NaN, or a query that is
    not finite, keep their bits."""
    G.require_gpu()
    for P in (16, 64):
        for D in (64, 128, 256):
            b = R.Batch([100], [61], P, 1, D, seed=2)
            q = _queries(b.T, hq, D, BF16, 1)
            clean = _call(b, q)
            for bad in (float("nan"), float("inf"), float("-inf")):
                q2 = q.clone()
                q2[70, 1, 5] = bad
                got = _call(b, q2)
                assert bool(torch.isnan(got[70, 1]).all())
                got[70, 1] = clean[70, 1]
                assert torch.equal(got, clean)
            for scales in (b.k_scales, b.v_scales):
                page = int(b.table[0, 128 // P])
                was = scales[page, 0].clone()
                scales[page, 0] = float("nan")
                got = _call(b, q)
                first = 128 - 61               # the first row that sees position 128
                assert bool(torch.isnan(got[first:]).all())
                assert torch.equal(got[:first], clean[:first])
                scales[page, 0] = was


@pytest.mark.parametrize("hq", [2, 32])
def test_sizes_of_queries_many_rows(hq):
    G.require_gpu()
    for dtype, sizes in ((F16, (6e-8, 1e-4, 3000.0)), (BF16, (1e-38, 1e-10, 1e15))):
        for size in sizes:
            b = R.Batch([70], [100], 32, 1, 64, seed=3)
            b.k_scales = torch.full_like(b.k_scales, 2.0 ** -10)
            q = (_queries(70, hq, 64, torch.float32, 6) * size).to(dtype)
            _check(b, q, scale=min(1.0, 0.1 / size))


def test_max_tokens_only_chooses():
    """Wrong bounds of the tokens give other kernels, not other rows."""
    G.require_gpu()
    b = R.Batch([90, 1, 20], [100, 300, 0], 32, 2, 64, seed=4)
    q = _queries(b.T, 4, 64, BF16, 2)
    for most in (None, 1, 90, 10 ** 6):
        _check(b, q, max_tokens=most)


def test_sizes_of_queries():
    """Queries at both ends of their type's range."""
    G.require_gpu()
    for dtype, sizes in ((F16, (6e-8, 1e-4, 3000.0)), (BF16, (1e-38, 1e-10, 1e15))):
        for size in sizes:
            b = R.Batch([1, 1], [100, 7], 32, 1, 64, seed=3)
            b.k_scales = torch.full_like(b.k_scales, 2.0 ** -10)
            q = _queries(2, 2, 64, F16 if dtype is F16 else torch.float32, 6, size if dtype is BF16 else 1.0)
            q = (q * size).to(dtype) if dtype is F16 else q.to(dtype)
            _check(b, q, scale=min(1.0, 0.1 / size))


def test_not_finite():
    """A query that is not finite spoils its row; a NaN scale the rows that see a
    token of its page; keys behind a row's position do not matter."""
    G.require_gpu()
    for P in (16, 64):
        b = R.Batch([4, 1], [61, 40], P, 2, 64, seed=2)
        q = _queries(b.T, 4, 64, F16, 1)
        clean = _call(b, q)
        for bad in (float("nan"), float("inf")):
            q2 = q.clone()
            q2[2, 3, 5] = bad
            got = _call(b, q2)
            assert bool(torch.isnan(got[2, 3]).all())
            got[2, 3] = clean[2, 3]
            assert torch.equal(got, clean)
        # the last page holds positions 64 and up: the last row alone sees it
        for scales in (b.k_scales, b.v_scales):
            page = int(b.table[0, 64 // P])
            was = scales[page, 1].clone()
            scales[page, 1] = float("nan")
            got = _call(b, q)
            assert bool(torch.isnan(got[3, 2:]).all())
            got[3, 2:] = clean[3, 2:]
            assert torch.equal(got, clean)
            scales[page, 1] = was
        # bytes and scales behind the last token: pages of the table that no token has reached
        wide = R.Batch([4, 1], [61, 40], P, 2, 64, seed=2, width=9, spare=2)
        for s in range(2):
            for i in range(-(-int(wide.lengths[s]) // P), 9):
                wide.table[s, i] = wide.pages - 1
        used = {int(p) for s in range(2) for p in wide.table[s, :-(-int(wide.lengths[s]) // P)]}
        free = [p for p in range(wide.pages) if p not in used]
        wide.table[wide.table == wide.pages - 1] = free[-1]
        if wide.pages - 1 in used:
            for s in range(2):
                for i in range(-(-int(wide.lengths[s]) // P)):
                    if wide.table[s, i] == free[-1]:
                        wide.table[s, i] = wide.pages - 1
        wide.k_scales[free], wide.v_scales[free] = float("nan"), float("inf")
        want, tol = R.attention(wide, q, 64 ** -0.5)
        R.check_rows(_call(wide, q), want, tol, F16)


def test_pages_and_lengths_without_sense():
    G.require_gpu()
    P = 16
    b = R.Batch([2, 3, 1, 2], [100, 50, 0, 30], P, 2, 64, seed=9, extra=2)
    b.table[0, 2] = -1                    # passed over
    b.table[1, 0] = b.pages
    b.table[1, 3] = 2 ** 31 - 1
    b.table[3] = -5                       # no usable page: rows of zeros
    b.lengths[2] = 0                      # its token stands before position 0
    q = _queries(b.T, 4, 64, BF16, 2)
    got = _check(b, q)
    assert bool((got[5] == 0).all()) and bool((got[6:8] == 0).all())
    b = R.Batch([2, 3], [100, 50], P, 2, 64, seed=9)
    b.lengths[0] = b.width * P + 50       # behind the table: what it names is read
    _check(b, _queries(b.T, 4, 64, F16, 3))
    q = _queries(b.T, 4, 64, F16, 3)
    for lengths, starts in (([-3, 2 ** 31 - 1], [0, 2, 5]), ([90, 50], [0, 10 ** 6, 1]), ([0, 0], [-9, 3, 4])):
        b.lengths[:], b.starts[:] = torch.tensor(lengths), torch.tensor(starts)
        _call(b, q)


def test_strides_streams_and_workspaces():
    """Rows further apart than their width, in both directions; raw stream
    handles; a workspace of the caller's; equal calls give equal bits."""
    G.require_gpu()
    b = R.Batch([1, 3, 1], [700, 20, 64], 32, 2, 128, seed=3)
    q = _queries(b.T, 8, 128, BF16, 9)
    want = _check(b, q)
    args = b.cuda()
    big = torch.full((b.T, 20, 128), 5.0, dtype=BF16, device="cuda")
    big[:, 3:11] = q.cuda()
    ws = torch.empty(mnb.mnb_attention_workspace(b.T, b.S, 8, 2, 128), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        big[:, 11:19] = 5.0
        torch.cuda.synchronize()
        mnb.attention_int8(big[:, 3:11], *args, big[:, 11:19], workspace=ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(big[:, 11:19].cpu(), want)
        assert bool((big[:, :3] == 5.0).all()) and bool((big[:, 19:] == 5.0).all())
        assert torch.equal(big[:, 3:11].cpu(), q)


@pytest.mark.parametrize("new,hq", [([1, 2, 1, 0], 6), ([1, 40, 3, 30], 6), ([1, 40, 3, 30], 40)],
                         ids=["few", "more", "many"])
def test_captured(new, hq):
    """A captured call replayed with other lengths, pages and queries, eager calls
    between the replays."""
    G.require_gpu()
    sets = []
    for i, before in enumerate(([500, 3, 60, 9], [0, 0, 0, 0], [1, 2500, 64, 0])):
        b = R.Batch(new, before, 16, 2, 64, seed=i, width=160, spare=2)
        pages = 400
        for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
            t = getattr(b, name)
            setattr(b, name, torch.cat((t, t.new_zeros((pages - t.shape[0],) + t.shape[1:]))))
        b.pages = pages
        sets.append((b, _queries(b.T, hq, 64, F16, i)))
    args, q = sets[0][0].cuda(), sets[0][1].cuda()
    out = torch.empty_like(q)
    mnb.attention_int8(q, *args, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mnb.attention_int8(q, *args, out)
    for i in (1, 2, 0, 2):
        b, x = sets[i]
        for dst, src in zip(args, b.index() + b.cache()):
            dst.copy_(src)
        q.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), _call(b, x))
        want, tol = R.attention(b, x, 64 ** -0.5)
        R.check_rows(out.cpu(), want, tol, F16)


def test_queries_of_every_size():
    """Queries up to bf16's largest value, and the smallest ones that scores can show."""
    G.require_gpu()
    for size, step in ((1e38, -124), (1e-28, 100)):
        for new, hq in (([1, 2], 2), ([70], 2), ([70], 30)):
            b = R.Batch(new, [40] * len(new), 32, 1, 64, seed=5)
            b.k_scales = torch.full_like(b.k_scales, 2.0 ** step)
            q = (_queries(b.T, hq, 64, torch.float32, 6).clamp(-3, 3) * size).to(BF16)
            mean = size * 2.0 ** step * 64 * 8      # of a score's magnitude
            _check(b, q, scale=3.0 / mean)


def test_starts_that_overlap():
    """Sequences that claim the same rows, more of them than the sizes of the call
    can hold: nothing behind the workspace, no row outside the sequences."""
    G.require_gpu()
    for T, G_ in ((150, 2), (40, 1), (150, 16)):
        b = R.Batch([T], [100], 32, 1, 64, seed=6, extra=4)
        b.S, b.table = 5, b.table.repeat(5, 1).contiguous()
        b.lengths = b.lengths.repeat(5)
        b.starts = torch.tensor([0, T, 0, T, 0, T], dtype=torch.int32)
        need = mnb.mnb_attention_workspace(b.T, b.S, G_, 1, 64)
        ws = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
        got = _call(b, _queries(b.T, G_, 64, BF16, 1), workspace=ws)
        assert bool((ws[need:] == 0x5A).all())
        assert bool((got[T:] == 9.0).all())


def test_no_pages():
    """A cache of no pages, a page table of no width: rows of zeros."""
    G.require_gpu()
    for new, hq in (([1, 3], 2), ([90, 1], 2), ([90, 1], 30)):
        for width in (0, 2):
            b = R.Batch(new, [10, 10], 16, 1, 64, seed=1)
            b.pages, b.width = 0, width
            b.table = torch.zeros(2, width, dtype=torch.int32)
            for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
                setattr(b, name, getattr(b, name)[:0])
            assert bool((_call(b, _queries(b.T, hq, 64, F16, 1)) == 0).all())


MANY = [
    # new, before, P, query heads, heads, D
    ([1 + i % 2 for i in range(70)], [3 * i for i in range(70)], 16, 4, 2, 64),
    ([i % 3 for i in range(131)], [(17 * i) % 90 for i in range(131)], 32, 8, 1, 128),
    ([66 if i % 9 == 0 else 1 for i in range(80)], [i for i in range(80)], 16, 2, 1, 64),
    ([1100, 1, 2], [0, 300, 7], 64, 64, 1, 64),      # row tiles enough for 64-bit counts
    ([70 if i == 4400 else 1 for i in range(4500)], [i % 3 for i in range(4500)], 16, 4, 1, 64),
]


@pytest.mark.parametrize("shape", MANY, ids=[str(i) for i in range(len(MANY))])
def test_many_sequences(shape):
    """More sequences than a wave has lanes, or more work than 32 bits count."""
    G.require_gpu()
    new, before, P, hq, heads, D = shape
    b = R.Batch(new, before, P, heads, D, seed=11, extra=2)
    q = _queries(b.T, hq, D, BF16, 5)
    for most in (None, max(new)):
        _check(b, q, max_tokens=most)


def test_more_tiles_than_a_grid_row():
    """2049 sequences of 64 tokens with 64 rows each: 65568 tiles."""
    G.require_gpu()
    b = R.Batch([64, 64, 64], [0, 0, 0], 64, 1, 64, seed=12)
    q = _queries(b.T, 64, 64, F16, 3)
    want = _check(b, q)
    times = 683
    big = R.Batch([64, 64, 64], [0, 0, 0], 64, 1, 64, seed=12)
    big.S, big.table, big.lengths = 3 * times, b.table.repeat(times, 1), b.lengths.repeat(times)
    big.starts = torch.arange(0, 64 * (3 * times + 1), 64, dtype=torch.int32)
    x = q.cuda().repeat(times, 1, 1)
    out = torch.full_like(x, 9.0)
    mnb.attention_int8(x, *big.cuda(), out)
    torch.cuda.synchronize()
    assert bool((out.view(times, 192, 64, 64) == out[:192]).all())
    exact, tol = R.attention(b, q, 64 ** -0.5)
    R.check_rows(out[:192].cpu(), exact, tol, F16)
    assert want.shape == out[:192].shape


def test_offsets_past_32_bits():
    """Pages more than 4 GiB into the cache."""
    G.require_gpu()
    pages, P, heads, D = 70000, 64, 8, 128
    for new in ([1, 2], [70, 1]):
        b = R.Batch(new, [200, 90], P, heads, D, seed=3)
        q = _queries(b.T, 16, D, BF16, 3)
        want = _call(b, q)
        where = torch.tensor([pages - 1 - 7 * i for i in range(b.pages)])
        dev = b.cuda()
        far = [torch.zeros((pages,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in dev[3:]]
        for dst, src in zip(far, dev[3:]):
            dst[where.cuda()] = src
        table = torch.where(b.table >= 0, where[b.table.clamp(min=0).long()], b.table.long()).to(torch.int32)
        out = torch.empty_like(q).cuda()
        mnb.attention_int8(q.cuda(), dev[0], dev[1], table.cuda(), *far, out)
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)


def test_two_graphs_of_one_workspace():
    """Two captured calls of different batches that share a workspace, replayed in
    turn with eager calls between them."""
    G.require_gpu()
    sets = []
    for i, new in enumerate(([1, 2, 1], [1, 400, 3])):
        b = R.Batch(new, [500, 30, 9], 16, 2, 64, seed=i)
        sets.append((b, _queries(b.T, 6, 64, F16, i)))
    need = max(mnb.mnb_attention_workspace(b.T, b.S, 6, 2, 64) for b, _ in sets)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    work = []
    for b, q in sets:
        args, x = b.cuda(), q.cuda()
        out = torch.empty_like(x)
        mnb.attention_int8(x, *args, out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mnb.attention_int8(x, *args, out, workspace=ws)
        work.append((graph, args, x, out, _call(b, q)))
    for i in (0, 1, 1, 0, 1, 0):
        graph, args, x, out, want = work[i]
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)
        _call(*sets[1 - i])


def test_scales_change_under_the_diagonal():
    """Value scales that change from page to page where some waves of a tile see no
    key any more: all waves stage the values in the same unit."""
    G.require_gpu()
    for D in (64, 128, 256):
        for P, before in ((16, 5), (16, 700), (64, 1), (64, 37), (256, 1), (256, 130)):
            b = R.Batch([333], [before], P, 2, D, seed=D + P)      # 1332 rows a key head
            for i in range(b.width):
                b.v_scales[int(b.table[0, i])] = 2.0 ** (-4 - 3 * (i % 4))
            _check(b, _queries(b.T, 8, D, BF16, 4))
