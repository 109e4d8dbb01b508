"""moe_nbits on the GPU against the formula in 64 bits on the CPU.

Bound of the error of one output, derived from the call's documented
roundings (u = 2^-24, the half step of fp32; every absolute sum is taken over
the same terms as the sum itself):

* gate and up: fp32 sums of exact products over H terms, in any order: at most
  H/32 block results plus the terms of one block and the reductions over lanes
  and waves meet in one chain, so |dg| <= (H/32 + 64) u sum|x w| =: Dg (Du
  alike).
* silu(g) u: |silu'| <= 1.1, and its own evaluation (exp, division, two
  products) is off by at most (|g| + 8) 2 u relative:
  dh <= 1.1 Dg |u| + |silu(g)| Du + 1.1 Dg Du + (|g| + 8) 2 u |h|.
* h is held in fp16 with a power-of-two scale per block of 32: 2^-11 |h|, and
  2^-25 of the block's largest where it falls below fp16's normal numbers.
* down: Dy = sum (dh + 2^-11 |h| + 2^-25 max) |w| + (I/32 + 64) u sum |h w|.
* p_j: exp of a difference of logits, a sum of at most E terms and a division:
  relative (|l - max| + E + 8) 2 u.
* the sum over top_k experts: top_k u of its absolute sum; the rounding of the
  result: eps/2 |y| + 2^-25 (below fp16's normal numbers).
"""
import numpy as np
import pytest
import torch

import block_wise_int4_matmulnbits_amd as mnb
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -24
INF = float("inf")


def _matrix(g, E, N, K, asym, lo=0.002, hi=0.02):
    B = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    S = (torch.rand(E, N, K // 32, generator=g) * (hi - lo) + lo).to(F16)
    Z = torch.randint(0, 256, (E, N, (K // 32 + 1) // 2), generator=g, dtype=torch.uint8) if asym else None
    return B, S, Z


def _layer(E, H, I, asym=True, seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    return _matrix(g, E, 2 * I, H, asym, **kw), _matrix(g, E, H, I, asym, **kw)


def _tokens(T, H, E, dtype, ldtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, generator=g).to(dtype), (torch.randn(T, E, generator=g) * 1.5).to(ldtype)


def _values(w, e):
    B, S, Z = (None if a is None else a[e] for a in w)
    N, nb = S.shape
    q = torch.stack((B & 15, B >> 4), -1).reshape(N, nb, 32).double()
    z = 8.0 if Z is None else torch.stack((Z & 15, Z >> 4), -1).reshape(N, -1)[:, :nb, None].double()
    return ((q - z) * S[:, :, None].double()).reshape(N, nb * 32)


def _route_ref(logits, k, renormalize):
    """ids [T, k] and weights [T, k] by the documented rules."""
    l = logits.double().numpy()
    T, E = l.shape
    ids, p = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        if np.isnan(l[t]).any() or (l[t] == np.inf).any():
            p[t] = np.nan
            continue
        order = [e for e in sorted(range(E), key=lambda e: (-l[t, e], e)) if l[t, e] > -np.inf][:k]
        if not order:
            continue
        over = l[t, order] if renormalize else l[t]
        w = np.exp(l[t, order] - l[t].max()) / np.exp(over - l[t].max()).sum()
        ids[t, :len(order)] = order
        p[t, :len(order)] = w
    return ids, p


def _moe_ref(x, ids, p, w1, w2):
    """(y, bound) in 64 bits, for the routing (ids, p); the bound excludes the
    rounding of the result."""
    T, H = x.shape
    I = w2[0].shape[2] * 2
    E = w2[0].shape[0]
    xd = x.to(F16).double()
    y, bound = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    total = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        W1, W2 = _values(w1, e), _values(w2, e)
        a = xd[t]
        gu, D = a @ W1.t(), (a.abs() @ W1.abs().t()) * (H / 32 + 64) * U
        g, u, Dg, Du = gu[:, :I], gu[:, I:], D[:, :I], D[:, I:]
        s = g * torch.sigmoid(g)
        h = s * u
        dh = 1.1 * Dg * u.abs() + s.abs() * Du + 1.1 * Dg * Du + (g.abs() + 8) * 2 * U * h.abs()
        top = (h.abs() + dh).reshape(len(t), -1, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(h.shape)
        dh = dh + 2.0 ** -11 * (h.abs() + dh) + 2.0 ** -25 * top
        yy, dy = h @ W2.t(), dh @ W2.abs().t() + (h.abs() + dh) @ W2.abs().t() * (I / 32 + 64) * U
        pp = torch.from_numpy(p[t, j])[:, None]
        rel = (40.0 + E + 8) * 2 * U
        y[t] += pp * yy
        bound[t] += pp * dy + pp * rel * (yy.abs() + dy)
        total[t] += pp * (yy.abs() + dy)
    return y, bound + ids.shape[1] * U * total


def _run(x, logits, w1, w2, k, renormalize, out_dtype, stream=None, workspace=None):
    T, H = x.shape
    out = torch.full((T * H + 16,), -1, dtype=torch.int16, device="cuda")
    ids = torch.full((T * k + 4,), -7, dtype=torch.int32, device="cuda")
    p = torch.full((T * k + 4,), -7.0, device="cuda")
    mnb.moe_nbits(x, logits, *w1, *w2, out[:T * H].view(out_dtype).view(T, H), k, renormalize=renormalize,
                  expert_ids=ids[:T * k].view(T, k), expert_weights=p[:T * k].view(T, k), workspace=workspace,
                  stream=stream)
    torch.cuda.synchronize()
    assert (out[T * H:] == -1).all() and (ids[T * k:] == -7).all() and (p[T * k:] == -7).all()
    return out[:T * H].view(out_dtype).view(T, H).cpu(), ids[:T * k].view(T, k).cpu(), p[:T * k].view(T, k).cpu()


def _cuda(w):
    return tuple(None if a is None else a.cuda() for a in w)


def _check(x, logits, w1, w2, k, renormalize, out_dtype, got):
    out, ids, p = got
    rids, rp = _route_ref(logits, k, renormalize)
    assert np.array_equal(ids.numpy(), rids)
    bad = np.isnan(rp)
    assert np.array_equal(p.isnan().numpy(), bad)
    spread = np.where(bad, 0, 40.0) + logits.shape[1] + 8
    assert (np.abs(p.double().numpy() - rp)[~bad] <= (spread * 2 * U * rp + 1e-38)[~bad]).all()
    y, bound = _moe_ref(x, rids, rp, w1, w2)
    ok = ~torch.from_numpy(bad.any(axis=1))
    tol = bound + torch.finfo(out_dtype).eps / 2 * (y.abs() + bound) + 2.0 ** -25
    err = (out.double() - y).abs()
    assert out[~ok].isnan().all()
    assert bool((err <= tol)[ok].all()), "worst %g of its tolerance" % float((err / tol)[ok].nan_to_num(9e9).max())
    nothing = torch.from_numpy((rids < 0).all(axis=1)) & ok
    assert bool((out[nothing] == 0).all())
    # On average the error lies far below the bound: a wrong block shows here.
    scale = y[ok].pow(2).mean().sqrt()
    if ok.any() and float(scale) > 0:
        rms = (out.double() - y)[ok].pow(2).mean().sqrt() / scale
        assert float(rms) <= torch.finfo(out_dtype).eps, float(rms)


CASES = [  # T, H, I, E, k
    (1, 32, 32, 1, 1), (1, 64, 96, 4, 2), (1, 1024, 512, 16, 8), (2, 96, 64, 3, 3), (3, 1056, 416, 10, 3),
    (4, 2048, 768, 8, 2), (5, 544, 64, 512, 16), (7, 160, 1120, 6, 4), (8, 4096, 96, 4, 1), (9, 128, 2080, 5, 5),
    (12, 256, 4128, 3, 2), (16, 512, 256, 4, 4), (17, 288, 160, 2, 1), (31, 800, 96, 12, 6), (33, 128, 544, 5, 5),
    (48, 192, 128, 1, 1), (64, 256, 160, 8, 2), (64, 64, 32, 128, 8), (64, 480, 1024, 2, 2), (40, 32, 64, 3, 1),
    (3, 65536, 32, 2, 1), (3, 32, 65536, 2, 2), (20, 65536, 32, 2, 1), (34, 32, 65536, 2, 2), (26, 1408, 2048, 4, 2),
    (64, 32, 32, 512, 16),
]


@pytest.mark.parametrize("T,H,I,E,k", CASES)
def test_layer(T, H, I, E, k):
    G.require_gpu()
    seed = T + H + I + E + k
    for dtype, ldtype, out_dtype, asym, renorm in ((F16, F32, BF16, True, True), (BF16, BF16, F16, False, False)):
        kw = dict(lo=0.002, hi=0.02) if max(H, I) < 8192 else dict(lo=1e-4, hi=1e-3)
        w1, w2 = _layer(E, H, I, asym, seed, **kw)
        x, logits = _tokens(T, H, E, dtype, ldtype, seed + 1)
        got = _run(x.cuda(), logits.cuda(), _cuda(w1), _cuda(w2), k, renorm, out_dtype)
        _check(x, logits, w1, w2, k, renorm, out_dtype, got)


@pytest.mark.parametrize("T,E,k", [(1, 7, 3), (6, 64, 8), (64, 10, 4), (13, 130, 16)])
def test_routing_ties_masks_and_bad_logits(T, E, k):
    """Equal logits go to the lower expert; -inf is never selected; a token
    with fewer experts left than k, with none, with +inf or NaN."""
    G.require_gpu()
    H, I = 64, 32
    w1, w2 = _layer(E, H, I, True, 3)
    x, _ = _tokens(T, H, E, F16, F32, 4)
    g = torch.Generator().manual_seed(5)
    for ldtype in (F32, F16, BF16):
        for renorm in (True, False):
            logits = torch.randint(-2, 3, (T, E), generator=g).to(ldtype)
            logits[torch.rand(T, E, generator=g) < 0.6] = -INF
            if T >= 6:
                logits[0] = -INF
                logits[1] = torch.finfo(ldtype).min
                logits[2] = 0
                logits[3, E // 2] = INF
                logits[4, E - 1] = float("nan")
                logits[5] = -INF
                logits[5, E - 1] = torch.finfo(ldtype).min
            got = _run(x.cuda(), logits.cuda(), _cuda(w1), _cuda(w2), k, renorm, F16)
            _check(x, logits, w1, w2, k, renorm, F16, got)


def test_zeros_of_both_signs_tie():
    """-0 and +0 are equal logits: the lower expert goes first."""
    G.require_gpu()
    E, k, T = 70, 3, 4
    w1, w2 = _layer(E, 64, 32, True, 3)
    x, _ = _tokens(T, 64, E, F16, F32, 4)
    for ldtype in (F32, F16, BF16):
        logits = torch.full((T, E), -1.0)
        logits[0, [5, 9, 68]] = torch.tensor([-0.0, 0.0, 0.0])
        logits[1, [5, 9, 68]] = torch.tensor([0.0, -0.0, 0.0])
        logits[2, [2, 66, 67, 69]] = torch.tensor([0.0, -0.0, 0.0, -0.0])
        logits[3] = -0.0
        logits = logits.to(ldtype)
        got = _run(x.cuda(), logits.cuda(), _cuda(w1), _cuda(w2), k, True, F16)
        assert got[1].tolist() == [[5, 9, 68], [5, 9, 68], [2, 66, 67], [0, 1, 2]]
        _check(x, logits, w1, w2, k, True, F16, got)


@pytest.mark.parametrize("T,E,k", [(3, 6, 2), (7, 6, 2), (30, 6, 2), (64, 6, 2)])
def test_tokens_that_are_not_finite_stay_alone(T, E, k):
    """Padding tokens (no expert) of NaN give zeros, a routed token of infinities
    a row that is not finite, and every other token the bits it has without
    them."""
    G.require_gpu()
    w1, w2 = (_cuda(w) for w in _layer(E, 96, 160, True, T))
    for dtype in (F16, BF16):
        x, logits = _tokens(T, 96, E, dtype, F32, T + 1)
        pads, hot = [0, T // 2], T - 1
        logits[pads] = -INF
        plain = _run(x.cuda(), logits.cuda(), w1, w2, k, True, BF16)
        x[pads], x[hot] = float("nan"), INF
        got = _run(x.cuda(), logits.cuda(), w1, w2, k, True, BF16)
        others = [t for t in range(T) if t != hot]
        assert torch.equal(got[0][others], plain[0][others]) and bool((got[0][pads] == 0).all())
        assert not bool(got[0][hot].isfinite().any())
        assert torch.equal(got[1], plain[1]) and torch.equal(got[2], plain[2])


def test_every_token_at_one_expert():
    """All tokens select the same experts: 64 rows at one expert."""
    G.require_gpu()
    for T in (1, 4, 5, 8, 15, 16, 17, 32, 63, 64):
        w1, w2 = _layer(4, 288, 224, True, T)
        x, _ = _tokens(T, 288, 4, BF16, F32, T)
        logits = torch.tensor([[0.0, 2.0, -1.0, 1.0]]).repeat(T, 1)
        got = _run(x.cuda(), logits.cuda(), _cuda(w1), _cuda(w2), 2, True, BF16)
        _check(x, logits, w1, w2, 2, True, BF16, got)


def test_intermediate_past_fp16():
    """silu(g) u far above fp16's largest number, and far below its smallest."""
    G.require_gpu()
    for factor, out_dtype, T in ((6.0, BF16, 5), (2.0 ** -13, BF16, 5), (6.0, BF16, 30), (2.0 ** -13, BF16, 30)):
        w1, w2 = _layer(2, 256, 128, True, 1, lo=0.1 * factor, hi=1.0 * factor)
        x, logits = _tokens(T, 256, 2, F16, F32, 2)
        x = x * (8 if factor > 1 else 2.0 ** -4)
        out, ids, p = _run(x.cuda(), logits.cuda(), _cuda(w1), _cuda(w2), 1, True, out_dtype)
        rids, rp = _route_ref(logits, 1, True)
        y, bound = _moe_ref(x, rids, rp, w1, w2)
        tol = bound + 2.0 ** -8 * (y.abs() + bound)
        assert bool(((out.double() - y).abs() <= tol).all())
        assert out.isfinite().all()


def test_poison_behind_every_array():
    """NaN scales and 0xFF bytes in front of and behind every array and in the
    experts that no token selects: nothing of it may show."""
    G.require_gpu()
    for T, H, I, E, k in ((3, 96, 160, 5, 2), (1, 1056, 416, 3, 1), (9, 352, 96, 4, 2), (20, 352, 96, 4, 2),
                          (40, 1056, 416, 3, 1)):
        w1, w2 = _layer(E, H, I, True, 8)
        x, logits = _tokens(T, H, E, F16, F32, 9)
        logits[:, E - 1] = -INF
        for B, S, Z in (w1, w2):
            B[E - 1], Z[E - 1] = 255, 255
            S[E - 1] = float("nan")

        def guarded(t, pad):
            raw = t.contiguous().view(torch.uint8).reshape(-1)
            buf = torch.full((raw.numel() + 2 * pad,), 255, dtype=torch.uint8, device="cuda")
            buf[pad:pad + raw.numel()] = raw.cuda()
            return buf[pad:pad + raw.numel()].view(t.dtype).view(t.shape)

        pads = (256, 258, 257)      # weights on 16 bytes, scales on 2, zero points anywhere
        g1 = tuple(guarded(t, p) for t, p in zip(w1, pads))
        g2 = tuple(guarded(t, p) for t, p in zip(w2, pads))
        got = _run(guarded(x, 256), guarded(logits, 4), g1, g2, k, True, F16)
        ref = _run(x.cuda(), logits.cuda(), _cuda(w1), _cuda(w2), k, True, F16)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert got[0].isfinite().all()
        _check(x, logits, w1, w2, k, True, F16, got)


@pytest.mark.parametrize("T,H,I,E,k", [(6, 512, 256, 16, 4), (24, 512, 256, 16, 4), (33, 512, 256, 4, 2)])
def test_streams_graph_and_workspace(T, H, I, E, k):
    """Two streams at once, two graphs (each with its own workspace) replayed
    together with changing tokens between eager calls, a dirty workspace of
    exactly the stated size."""
    G.require_gpu()
    w1, w2 = (_cuda(w) for w in _layer(E, H, I, True, 1))
    data = [tuple(t.cuda() for t in _tokens(T, H, E, BF16, F32, 30 + i)) for i in range(4)]
    want = [_run(x, l, w1, w2, k, True, F16) for x, l in data]
    need = mnb.mnb_moe_workspace(T, H, I, E, k)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    c0 = mnb.mnb_counters_get()
    for (x, l), w in zip(data, want):
        assert all(torch.equal(a, b) for a, b in zip(_run(x, l, w1, w2, k, True, F16, workspace=ws[:need]), w))
    c1 = mnb.mnb_counters_get()
    assert c1["calls"] == c0["calls"] + 4
    assert (ws[need:] == 255).all()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(T, H, dtype=F16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for i, (x, l) in enumerate(data):
        mnb.moe_nbits(x, l, *w1, *w2, outs[i], k, stream=streams[i % 2])
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.cpu(), w[0])
    x_in, l_in = (t.clone() for t in data[0])
    graphs = []
    for o in outs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mnb.moe_nbits(x_in, l_in, *w1, *w2, o, k)
        graphs.append(g)
    for i, (x, l) in enumerate(data):
        x_in.copy_(x)
        l_in.copy_(l)
        for o in outs[:2]:
            o.fill_(-1)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        nxt = (i + 1) % 4
        assert torch.equal(_run(*data[nxt], w1, w2, k, True, F16)[0], want[nxt][0])
        for o in outs[:2]:
            assert torch.equal(o.cpu(), want[i][0])


def test_offsets_past_32_bits():
    """Experts past 2^32 bytes of packed weights: 400 experts of 2 x 1376 rows
    of 8192; only the last ones are selected."""
    G.require_gpu()
    E, H, I, T, k = 400, 8192, 1376, 2, 2
    g = torch.Generator().manual_seed(2)
    w1 = (torch.full((E, 2 * I, H // 2), 255, dtype=torch.uint8, device="cuda"),
          torch.full((E, 2 * I, H // 32), float("nan"), dtype=F16, device="cuda"), None)
    w2 = (torch.full((E, H, I // 2), 255, dtype=torch.uint8, device="cuda"),
          torch.full((E, H, I // 32), float("nan"), dtype=F16, device="cuda"), None)
    assert w1[0].numel() > 1 << 32
    small = (_matrix(g, 3, 2 * I, H, False, 5e-4, 5e-3), _matrix(g, 3, H, I, False, 5e-4, 5e-3))
    for big, s in zip((w1, w2), small):
        big[0][E - 3:], big[1][E - 3:] = s[0].cuda(), s[1].cuda()
    x, _ = _tokens(T, H, E, F16, F32, 3)
    logits = torch.full((T, E), -INF)
    logits[:, E - 3:] = torch.tensor([[1.0, 0.5, -2.0], [-1.0, 2.0, 0.0]])
    out, ids, p = _run(x.cuda(), logits.cuda(), w1, w2, k, True, BF16)
    assert (ids >= E - 3).all()
    _check(x, logits[:, E - 3:].contiguous(), *small, k, True, BF16, (out, ids - (E - 3), p))


def test_binding_refusals():
    G.require_gpu()
    T, H, I, E, k = 3, 64, 96, 4, 2
    w1, w2 = (_cuda(w) for w in _layer(E, H, I, True, 1))
    x, l = (t.cuda() for t in _tokens(T, H, E, F16, F32, 2))
    out = torch.empty(T, H, dtype=F16, device="cuda")
    for args in ((x[:, :32].contiguous(), l, *w1, *w2, out, k), (x, l[:2], *w1, *w2, out, k),
                 (x, l[:, :3].contiguous(), *w1, *w2, out, k), (x, l, *w1[:2], w2[2], *w2, out, k),
                 (x, l, w1[0][:, :62].contiguous(), *w1[1:], *w2, out, k), (x, l, *w1, *w2, out[:2], k),
                 (x.cpu(), l, *w1, *w2, out, k), (x, l.t().contiguous().t(), *w1, *w2, out, k)):
        with pytest.raises(ValueError):
            mnb.moe_nbits(*args)
    with pytest.raises(TypeError):
        mnb.moe_nbits(x, l.double(), *w1, *w2, out, k)
    with pytest.raises(TypeError):
        mnb.moe_nbits(x.float(), l, *w1, *w2, out, k)
    with pytest.raises(ValueError):
        mnb.moe_nbits(x, l, *w1, *w2, out, k, expert_ids=torch.empty(T, 3, dtype=torch.int32, device="cuda"))
    for bad_k in (0, 5):
        with pytest.raises(mnb.MnbError):
            mnb.moe_nbits(x, l, *w1, *w2, out, bad_k)
    with pytest.raises(mnb.MnbError):
        mnb.moe_nbits(x, l, *w1, *w2, out, k, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
