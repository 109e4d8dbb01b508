"""The 8-bit and expert calls as programs make them: streams given as raw
handles, two host threads at once, the same tensor in two places."""
import threading

import pytest
import torch

import block_wise_int4_matmulnbits_amd as mnb
from tests import gpu_util as G
from tests import test_gpu_int8 as I8
from tests import test_gpu_moe as MOE

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _int8(seed):
    m, K, N = 70, 1024, 300            # a workspace and two launches
    _, _, W, b, bias = (t.cuda() for t in I8._inputs(1, K, N, seed))
    x = I8._rows(m, K, BF16, seed).cuda()
    return lambda out, stream=None: mnb.matmul_int8(x, None, W, b, bias, out, stream=stream), (m, N)


def _moe(seed, T=33):
    E, H, I, k = 4, 256, 160, 2        # five launches
    w1, w2 = (MOE._cuda(w) for w in MOE._layer(E, H, I, True, seed))
    x, logits = (t.cuda() for t in MOE._tokens(T, H, E, BF16, F32, seed))
    return lambda out, stream=None: mnb.moe_nbits(x, logits, *w1, *w2, out, k, stream=stream), (T, H)


@pytest.mark.parametrize("make", [_int8, _moe, lambda seed: _moe(seed, 3)], ids=["int8", "moe_wide", "moe_narrow"])
def test_raw_stream_handles(make):
    G.require_gpu()
    call, shape = make(1)
    want = call(torch.empty(shape, dtype=F16, device="cuda"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        out = torch.full(shape, float("nan"), dtype=F16, device="cuda")
        torch.cuda.synchronize()
        for _ in range(3):
            assert call(out, stream) is out
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_threads():
    """Each thread on a stream of its own, its calls back to back; a workspace
    shared between them would show."""
    G.require_gpu()
    calls = [_int8(1), _moe(2), _int8(3), _moe(4, 5)]
    want = []
    for call, shape in calls:
        want.append(call(torch.empty(shape, dtype=F16, device="cuda")))
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            call, shape = calls[i]
            outs = [torch.empty(shape, dtype=F16, device="cuda") for _ in range(40)]
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                for o in outs:
                    call(o)
            stream.synchronize()
            for o in outs:
                assert torch.equal(o, want[i])
        except BaseException as e:     # noqa: B902 (reported below)
            errors.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_same_tensor_twice():
    """Inputs may be one buffer; an output may not be an input."""
    G.require_gpu()
    W = torch.randint(-127, 128, (48, 64), dtype=torch.int8).cuda()
    s = (torch.rand(48) * 1e-2).cuda()
    out = torch.empty(48, 48, dtype=F16, device="cuda")
    mnb.matmul_int8(W, s, W, s, s, out)
    torch.cuda.synchronize()
    I8._check(out.cpu(), W.cpu(), s.cpu(), W.cpu(), s.cpu(), s.cpu(), F16)
    x = torch.randn(3, 64, device="cuda").to(F16)
    q, qs = torch.empty(3, 64, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    with pytest.raises(mnb.MnbError):
        mnb.quantize_rows_int8(x, x.view(torch.int8).view(-1)[:192].view(3, 64), qs)
    mnb.quantize_rows_int8(x, q, qs)
    E, H, I, k = 3, 64, 64, 2
    w1, w2 = (MOE._cuda(w) for w in MOE._layer(E, H, I, True, 5))
    logits = torch.randn(3, E, device="cuda")
    with pytest.raises(mnb.MnbError):
        mnb.moe_nbits(x, logits, *w1, *w2, x, k)
    with pytest.raises(mnb.MnbError):
        mnb.moe_nbits(x, logits, *w1, *w2, torch.empty_like(x), k, workspace=x)
