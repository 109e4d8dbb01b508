"""Every kernel that the 8-bit products and the expert layer choose from, in
its steady state, against exact arithmetic (tests/test_quant_routes_host.py
asserts on the host which kernel each shape gets).

* Tiles of the 8-bit product: K so long that every slot of the ring of stages
  is filled at least twice with data that is used, with a ragged last stage and
  without.
* The kernel for few rows: one to eight units of K per wave, sixteen waves and
  eight, rows it quantises itself, and rows that do not fit the registers of
  the waves that quantise them.
* The expert layer: every variant of its first and second launch.
"""
import numpy as np
import pytest
import torch

from tests import gpu_util as G
from tests import test_gpu_int8 as I8
from tests import test_gpu_moe as MOE
from tests import test_gpu_moe_range as RANGE

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32

TILES = [("256x256", 2049, 1040, 4100), ("256x256", 700, 1024, 12001), ("256x128", 257, 1040, 12001),
         ("256x128", 1000, 1152, 4100), ("128x128", 129, 2064, 9001), ("128x128", 500, 2048, 4100),
         ("128x64", 129, 2064, 5999), ("128x64", 257, 2048, 4100), ("64x64", 17, 2064, 9001), ("64x64", 40, 2304, 9001),
         ("64x32", 40, 4112, 4100), ("64x32", 2049, 4096, 100), ("32x32", 17, 6160, 33), ("32x32", 64, 6144, 100)]

ROWS = [(1, 6144, 70), (1, 8192, 70), (1, 10240, 33), (1, 12288, 70), (1, 14336, 70), (1, 16384, 70), (2, 16384, 17),
        (5, 6160, 50), (6, 4224, 40), (7, 4224, 40), (3, 10256, 19), (1, 2048, 5001), (16, 2048, 4201), (9, 1936, 4099),
        (1, 4096, 65601), (7, 4096, 65553)]

EXPERTS = [(1, 4096, 256, 8, 2), (2, 2048, 96, 8, 2), (24, 4096, 256, 8, 2), (24, 4096, 96, 8, 2), (24, 2048, 256, 8, 2),
           (24, 2048, 96, 8, 2), (12, 16384, 64, 2, 1), (3, 18464, 32, 2, 1), (12, 16416, 64, 2, 1), (6, 256, 64, 3, 3),
           (32, 352, 128, 8, 2), (32, 352, 256, 8, 2)]


@pytest.mark.parametrize("tile,m,K,N", TILES)
def test_tiles(tile, m, K, N):
    G.require_gpu()
    A, a, W, b, bias = I8._inputs(m, K, N, m + K + N, full=True)
    dev = [t.cuda() for t in (A, a, W, b, bias)]
    for out_dtype in (F16, BF16):
        out = I8._product(*dev, out_dtype)
        I8._check(out, A, a, W, b, bias, out_dtype)
        few = I8._product(dev[0][:5].contiguous(), dev[1][:5].contiguous(), *dev[2:], out_dtype)
        assert torch.equal(few.view(torch.int16), out[:5].view(torch.int16))


@pytest.mark.parametrize("m,K,N", ROWS)
def test_few_rows(m, K, N):
    """int8 rows, and fp16 and bf16 rows quantised in the call."""
    G.require_gpu()
    A, a, W, b, bias = I8._inputs(m, K, N, 3 * m + K + N, full=True)
    dev = [t.cuda() for t in (A, a, W, b, bias)]
    I8._check(I8._product(*dev, BF16), A, a, W, b, bias, BF16)
    for dtype in (F16, BF16):
        x = I8._rows(m, K, dtype, m + K)
        got = I8._product(x.cuda(), None, *dev[2:], F16)
        q, s = (torch.from_numpy(t) for t in I8._quantize_ref(x))
        I8._check(got, q, s, W, b, bias, F16)
        assert torch.equal(got.view(torch.int16), I8._product(q.cuda(), s.cuda(), *dev[2:], F16).view(torch.int16))


@pytest.mark.parametrize("T,H,I,E,k", EXPERTS)
def test_expert_kernels(T, H, I, E, k):
    G.require_gpu()
    kw = dict(lo=0.002, hi=0.02) if H < 8192 else dict(lo=1e-4, hi=1e-3)
    for dtype, ldtype, out_dtype, asym, renorm in ((F16, F32, BF16, True, True), (BF16, BF16, F16, False, False),
                                                   (BF16, F32, F16, True, True)):
        w1, w2 = MOE._layer(E, H, I, asym, T + H + I, **kw)
        x, logits = MOE._tokens(T, H, E, dtype, ldtype, T + H)
        got = MOE._run(x.cuda(), logits.cuda(), MOE._cuda(w1), MOE._cuda(w2), k, renorm, out_dtype)
        RANGE.check(x, logits, w1, w2, k, renorm, got, out_dtype)
