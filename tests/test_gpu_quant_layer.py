"""A layer of a quantised model as it is served: 8-bit projection (rows
quantised once, and by the call itself), router, 4-bit expert layer, 4-bit
head.  Every operator's output is checked against its own formula in 64 bits
on the inputs it got, and a captured step replayed with other tokens, with
eager work and synchronizations in between, gives the eager step's bits."""
import numpy as np
import pytest
import torch

import block_wise_int4_matmulnbits_amd as mnb
from tests import gpu_util as G
from tests import test_gpu_int8 as I8
from tests import test_gpu_moe as MOE

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


class Layer:
    def __init__(self, H, I, E, k, V, seed):
        g = torch.Generator().manual_seed(seed)
        self.H, self.I, self.E, self.k, self.V = H, I, E, k, V
        self.proj = torch.randint(-127, 128, (H, H), generator=g, dtype=torch.int8)
        self.proj_scales = torch.rand(H, generator=g) * 2e-4 + 1e-5
        self.bias = torch.randn(H, generator=g) * 0.1
        self.router = (torch.randn(H, E, generator=g) * 0.05)
        self.w1, self.w2 = MOE._layer(E, H, I, True, seed + 1, lo=5e-4, hi=5e-3)
        B, S, Z = MOE._matrix(g, 1, V, H, True, 5e-4, 5e-3)
        self.head = (B[0], S[0], Z[0])

    def cuda(self):
        for n in ("proj", "proj_scales", "bias", "router"):
            setattr(self, n, getattr(self, n).cuda())
        self.w1, self.w2, self.head = MOE._cuda(self.w1), MOE._cuda(self.w2), MOE._cuda(self.head)
        return self

    def step(self, x, bufs):
        """The served step; every intermediate stays in bufs."""
        mnb.quantize_rows_int8(x, bufs["q"], bufs["qs"])
        mnb.matmul_int8(bufs["q"], bufs["qs"], self.proj, self.proj_scales, self.bias, bufs["a"])
        mnb.matmul_int8(x, None, self.proj, self.proj_scales, self.bias, bufs["a2"])
        torch.add(x, bufs["a"], out=bufs["x2"])
        torch.matmul(bufs["x2"].float(), self.router, out=bufs["logits"])
        mnb.moe_nbits(bufs["x2"], bufs["logits"], *self.w1, *self.w2, bufs["m"], self.k, expert_ids=bufs["ids"],
                      expert_weights=bufs["p"])
        torch.add(bufs["x2"], bufs["m"], out=bufs["x3"])
        mnb.matmul_nbits(bufs["x3"], *self.head, bufs["out"])
        return bufs

    def buffers(self, T, dtype):
        dev = dict(device="cuda")
        b = {n: torch.empty(T, self.H, dtype=dtype, **dev) for n in ("a", "a2", "x2", "m", "x3")}
        b.update(q=torch.empty(T, self.H, dtype=torch.int8, **dev), qs=torch.empty(T, **dev),
                 logits=torch.empty(T, self.E, **dev), ids=torch.empty(T, self.k, dtype=torch.int32, **dev),
                 p=torch.empty(T, self.k, **dev), out=torch.empty(T, self.V, dtype=F16, **dev))
        return b


@pytest.mark.parametrize("T,E,k,dtype", [(1, 8, 2, BF16), (5, 8, 2, F16), (24, 8, 2, BF16), (64, 4, 2, F16)])
def test_layer_as_served(T, E, k, dtype):
    G.require_gpu()
    L = Layer(512, 288, E, k, 1000, 40 + T).cuda()
    g = torch.Generator().manual_seed(T)
    xs = [(torch.randn(T, L.H, generator=g)).to(dtype).cuda() for _ in range(3)]
    eager = []
    for x in xs:
        b = L.step(x, L.buffers(T, dtype))
        torch.cuda.synchronize()
        eager.append({n: t.clone() for n, t in b.items()})
        h = {n: t.cpu() for n, t in b.items()}
        rq, rs = I8._quantize_ref(x.cpu())
        assert np.array_equal(h["q"].numpy(), rq) and np.array_equal(h["qs"].numpy(), rs)
        assert torch.equal(h["a"].view(torch.int16), h["a2"].view(torch.int16))
        I8._check(h["a"], h["q"], h["qs"], L.proj.cpu(), L.proj_scales.cpu(), L.bias.cpu(), dtype)
        w1, w2 = (tuple(t.cpu() for t in w) for w in (L.w1, L.w2))
        MOE._check(h["x2"], h["logits"], w1, w2, k, True, dtype, (h["m"], h["ids"], h["p"]))
        # The head: fp32 sums of the exact products of the fp16 rows (decode),
        # or of weights rounded to fp16 (prefill: 2^-11 of each product).
        B, S, Z = (t.cpu()[None] for t in L.head)
        W = MOE._values((B, S, Z), 0)
        xd = h["x3"].to(F16).double()
        y, mag = xd @ W.t(), xd.abs() @ W.abs().t()
        tol = mag * (2.0 ** -11 + (L.H / 32 + 64) * 2.0 ** -24) + 2.0 ** -11 * y.abs() + 2.0 ** -24
        assert bool(((h["out"].double() - y).abs() <= tol).all())
    x_in, bufs = xs[0].clone(), L.buffers(T, dtype)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step(x_in, bufs)
    for i in (0, 1, 2, 1):
        x_in.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        for n in ("q", "qs", "a", "a2", "ids", "p", "m", "out"):
            assert torch.equal(bufs[n], eager[i][n]), n
        again = L.step(xs[(i + 1) % 3], L.buffers(T, dtype))
        torch.cuda.synchronize()
        assert torch.equal(again["out"], eager[(i + 1) % 3]["out"])
