"""moe_nbits over the whole range of its inputs, against the formula in 64 bits
on the CPU: bf16 activations far above and far below fp16's numbers, and
routing weights of logits that lie far apart.

Bound of the error of one output, from the call's documented roundings (u =
2^-24, the half step of fp32):

* x: fp16 rows are taken as they are.  bf16 rows are held in fp16 under a
  power of two that brings the largest value it serves to 2^14 .. 2^15.  A
  bf16 number has 8 significant bits, so what then lies above 2^-17 is exact
  and the rest is off by half of fp16's smallest step, 2^-25, which is at most
  2^-39 of the largest: dx <= 2^-39 max|x| over the row.
* gate and up: fp32 sums of exact products, D = (H/32 + 64) u sum|x w| +
  2^-39 max|x| sum|w|.
* silu(g) u: |silu'| <= 1.1; exp to 2 u, a sum, a division and two products:
  dh <= 1.1 Dg |u| + |silu(g)| Du + 1.1 Dg Du + 8 u |h|.
* h in fp16 under a power of two per block of 32, or per row where an expert
  sees eight tokens or more (tokens * top_k >= 8 * experts): 2^-11 |h| and
  2^-25 of the largest |h| under the same power.
* down: sum dh |w| + (I/32 + 64) u sum|h w|; the routing weights' error times
  |y|; top_k u of the sum over the experts; the rounding of the result.
"""
import numpy as np
import pytest
import torch

from tests import gpu_util as G
from tests import test_gpu_moe as MOE

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -24


def _reference(x, ids, p, w1, w2, dp):
    """(y, bound) in 64 bits; dp: relative error of the routing weights."""
    T, H = x.shape
    E, k = w2[0].shape[0], ids.shape[1]
    I = w2[0].shape[2] * 2
    wide = T * k >= 8 * E
    xd = x.double()
    y, bound, total = (torch.zeros(T, H, dtype=torch.float64) for _ in range(3))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        W1, W2 = MOE._values(w1, e), MOE._values(w2, e)
        a = xd[t]
        gu, D = a @ W1.t(), (a.abs() @ W1.abs().t()) * (H / 32 + 64) * U
        if x.dtype == BF16:
            D = D + 2.0 ** -39 * a.abs().amax(1, keepdim=True) * W1.abs().sum(1)
        g, u, Dg, Du = gu[:, :I], gu[:, I:], D[:, :I], D[:, I:]
        s = g * torch.sigmoid(g)
        h = s * u
        dh = 1.1 * Dg * u.abs() + s.abs() * Du + 1.1 * Dg * Du + 8 * U * h.abs()
        m = h.abs() + dh
        top = m.amax(1, keepdim=True) if wide else \
            m.reshape(len(t), -1, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(h.shape)
        dh = dh + 2.0 ** -11 * m + 2.0 ** -25 * top
        yy, dy = h @ W2.t(), dh @ W2.abs().t() + (h.abs() + dh) @ W2.abs().t() * (I / 32 + 64) * U
        pp = torch.from_numpy(p[t, j])[:, None]
        y[t] += pp * yy
        bound[t] += pp * (dy + dp * (yy.abs() + dy))
        total[t] += pp * (yy.abs() + dy)
    return y, bound + k * U * total


def check(x, logits, w1, w2, k, renormalize, got, out_dtype=BF16):
    """What a call with these inputs returned."""
    out, ids, p = got
    rids, rp = MOE._route_ref(logits, k, renormalize)
    assert np.array_equal(ids.numpy(), rids)
    # exp of differences of logits (up to 16, rounded to fp32), their sum, a division.
    dp = (16 + logits.shape[1] + 10) * U
    assert (np.abs(p.double().numpy() - rp) <= dp * rp).all()
    y, bound = _reference(x, rids, rp, w1, w2, dp)
    half, floor = torch.finfo(out_dtype).eps / 2, torch.finfo(out_dtype).smallest_normal
    tol = bound + half * (y.abs() + bound) + half * floor
    err = (out.double() - y).abs()
    assert bool((err <= tol).all()), "worst %g of its tolerance" % float((err / tol).nan_to_num(9e9).max())
    # On average the error lies far below the bound: a wrong block shows here.
    rms = float(((out.double() - y) / y.pow(2).mean(1, keepdim=True).sqrt()).pow(2).mean().sqrt())
    assert rms <= 2 * half, rms


# T, H, I, E, k: every token staged at once, the rows of a batch (four and
# eight), K staged in spans (four and eight rows), 16 and 32 rows.
KERNELS = [(1, 96, 64, 4, 2), (3, 96, 160, 5, 2), (6, 96, 64, 8, 2), (9, 352, 96, 4, 2), (3, 65536, 32, 2, 1),
           (12, 16384, 64, 2, 1), (32, 352, 96, 8, 2), (40, 1056, 416, 3, 1)]


@pytest.mark.parametrize("T,H,I,E,k", KERNELS)
@pytest.mark.parametrize("values", ["large", "small", "rows", "blocks", "elements"])
def test_bf16_range(T, H, I, E, k, values):
    """Tokens of about 1e6, of about 1e-7, of a size of their own, with blocks
    and single elements that differ by many powers of two."""
    G.require_gpu()
    kw = dict(lo=0.002, hi=0.02) if H < 8192 else dict(lo=1e-4, hi=1e-3)
    w1, w2 = MOE._layer(E, H, I, True, T + H, **kw)
    x, logits = MOE._tokens(T, H, E, F32, F32, T + H + 1)
    logits = logits.clamp(-4, 4)
    g = torch.Generator().manual_seed(T)
    if values == "large":
        x = x * 1e6
    elif values == "small":
        x = x * 1e-7
    elif values == "rows":
        x = x * torch.exp2(torch.randint(-40, 41, (T, 1), generator=g).float())
    elif values == "blocks":
        x = x * torch.exp2(torch.randint(-40, 21, (T, H // 32, 1), generator=g).float()).expand(-1, -1, 32).reshape(T, H)
        x[:, :32] = 0
    else:
        x = x * torch.exp2(torch.randint(-30, 21, (T, H), generator=g).float())
    x = x.to(BF16)
    got = MOE._run(x.cuda(), logits.cuda(), MOE._cuda(w1), MOE._cuda(w2), k, True, BF16)
    check(x, logits, w1, w2, k, True, got)


@pytest.mark.parametrize("T,E,k", [(1, 2, 2), (5, 8, 4), (20, 130, 16), (64, 3, 2)])
def test_routing_weights_of_distant_logits(T, E, k):
    """Logits on multiples of 1/8 up to 80 apart: their differences are exact in
    fp32, so p is off by exp's two half steps in the numerator and in every
    term of the sum, E additions and a division (five half steps at most)."""
    G.require_gpu()
    w1, w2 = (MOE._cuda(w) for w in MOE._layer(E, 64, 32, True, 3))
    x, _ = MOE._tokens(T, 64, E, F16, F32, 4)
    g = torch.Generator().manual_seed(E)
    logits = torch.randint(-320, 321, (T, E), generator=g).float() / 8
    for renormalize in (True, False):
        _, ids, p = MOE._run(x.cuda(), logits.cuda(), w1, w2, k, renormalize, F16)
        rids, rp = MOE._route_ref(logits, k, renormalize)
        assert np.array_equal(ids.numpy(), rids)
        rel = np.abs(p.double().numpy() - rp) / rp
        assert rel.max() <= (E + 9) * U, rel.max() / U
