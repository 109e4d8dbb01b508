"""moe_nbits: routing weights of logits that lie far apart, against exact
arithmetic (u = 2^-24, the half step of fp32)."""
import numpy as np
import pytest
import torch

from tests import gpu_util as G
from tests import test_gpu_moe as MOE

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -24


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
