"""Refusals, workspace sizes and empty calls of quantize_rows_int8,
matmul_int8 and moe_nbits, without a GPU: every check runs on the host before
anything is launched, so the addresses below are never dereferenced."""
import ctypes

import pytest

import block_wise_int4_matmulnbits_amd as mnb

P = 0x100000000   # buffers P, 2P, 3P, ...: disjoint, 16-byte aligned


def _status(call, args, status):
    c0 = mnb.mnb_counters_get()
    st = call(**args)
    assert st == status, mnb.mnb_status_string(st)
    assert mnb.mnb_counters_get() == c0
    assert mnb.mnb_status_string(st) != "unknown status"


def _quantize(A=P, a=mnb.MNB_F16, m=2, K=64, q=2 * P, s=3 * P):
    return mnb.lib().quantize_rows_int8(A, a, m, K, q, s, None)


@pytest.mark.parametrize("args,status", [
    (dict(m=-1), 6), (dict(m=(1 << 20) + 1), 6), (dict(K=-16), 2), (dict(K=8), 2), (dict(K=(1 << 24) + 16), 2),
    (dict(a=mnb.MNB_F32), 4), (dict(a=mnb.MNB_I8), 4), (dict(a=-1), 4), (dict(A=None), 1), (dict(q=None), 1),
    (dict(s=None), 1), (dict(A=P + 8), 5), (dict(q=2 * P + 4), 5), (dict(s=3 * P + 2), 5),
    (dict(q=P + 128), 8), (dict(s=P + 4), 8), (dict(s=2 * P + 124), 8),
])
def test_quantize_refusals(args, status):
    _status(_quantize, args, status)


def _int8(A=P, a=mnb.MNB_I8, sa=2 * P, m=3, K=64, N=5, B=3 * P, sb=4 * P, bias=None, out=5 * P, o=mnb.MNB_F16,
          ws=None, size=0):
    return mnb.lib().matmul_int8(A, a, sa, m, K, N, B, sb, bias, out, o, ws, size, None)


F16 = dict(a=mnb.MNB_F16, sa=None, ws=6 * P, size=1 << 24)


@pytest.mark.parametrize("args,status", [
    (dict(m=-1), 6), (dict(m=(1 << 20) + 1), 6), (dict(K=-16), 2), (dict(K=24), 2), (dict(K=131072), 2),
    (dict(N=-1), 2), (dict(N=1 << 31), 2), (dict(N=mnb.MNB_MAX_N_INT8 + 1), 2), (dict(a=mnb.MNB_F32), 4), (dict(a=4), 4), (dict(o=mnb.MNB_F32), 4),
    (dict(o=mnb.MNB_I8), 4), (dict(A=None), 1), (dict(sa=None), 1), (dict(B=None), 1), (dict(sb=None), 1),
    (dict(out=None), 1), (dict(A=P + 1), 5), (dict(B=3 * P + 8), 5), (dict(sa=2 * P + 2), 5),
    (dict(sb=4 * P + 1), 5), (dict(bias=7 * P + 2), 5), (dict(out=5 * P + 1), 5),
    (dict(out=P), 8), (dict(out=3 * P + 318), 8), (dict(out=2 * P), 8), (dict(out=4 * P), 8),
    (dict(bias=5 * P), 8),
])
def test_int8_refusals(args, status):
    _status(_int8, args, status)


def test_int8_workspace_refusals():
    m, K, N = 300, 4096, 4096
    need = mnb.mnb_int8_workspace(mnb.MNB_F16, m, K, N)
    assert need >= m * K
    base = dict(F16, m=m, K=K, N=N)
    _status(_int8, dict(base, size=need - 1), 11)
    _status(_int8, dict(base, ws=None), 1)
    _status(_int8, dict(base, ws=6 * P + 8), 5)
    _status(_int8, dict(base, ws=P + 64), 8)           # over the rows
    _status(_int8, dict(base, ws=5 * P + 64), 8)       # over the output
    assert mnb.mnb_int8_workspace(mnb.MNB_I8, m, K, N) == mnb.mnb_int8_workspace(mnb.MNB_I8, m, K, N)
    for bad in ((mnb.MNB_F32, m, K, N), (mnb.MNB_F16, -1, K, N), (mnb.MNB_F16, m, 8, N), (mnb.MNB_F16, m, K, -1),
                (mnb.MNB_F16, 0, K, N), (mnb.MNB_F16, m, K, 0)):
        assert mnb.mnb_int8_workspace(*bad) == 0


def _moe(x=P, xd=mnb.MNB_F16, T=3, l=2 * P, ld=mnb.MNB_F32, k=2, renorm=1, E=4, H=64, I=96, w1=3 * P, s1=4 * P,
         z1=5 * P, w2=6 * P, s2=7 * P, z2=8 * P, block=32, out=9 * P, o=mnb.MNB_BF16, ids=10 * P, pw=11 * P,
         ws=12 * P, size=1 << 24, weights=True):
    w = mnb.mnb_moe_weights(E, H, I, w1, s1, z1, w2, s2, z2, block)
    return mnb.lib().moe_nbits(x, xd, T, l, ld, k, renorm, ctypes.byref(w) if weights else None, out, o, ids, pw,
                               ws, size, None)


@pytest.mark.parametrize("args,status", [
    (dict(T=-1), 6), (dict(T=65), 6), (dict(k=0), 2), (dict(k=5), 2), (dict(k=17, E=32), 2), (dict(E=0), 2),
    (dict(E=513), 2), (dict(H=48), 2), (dict(H=0), 2), (dict(H=65568), 2), (dict(I=0), 2), (dict(I=33), 2),
    (dict(I=65568), 2), (dict(block=64), 3), (dict(xd=mnb.MNB_F32), 4), (dict(xd=mnb.MNB_I8), 4),
    (dict(o=mnb.MNB_F32), 4), (dict(ld=mnb.MNB_I8), 4), (dict(ld=-1), 4), (dict(weights=False), 1),
    (dict(x=None), 1), (dict(l=None), 1), (dict(w1=None), 1), (dict(s1=None), 1), (dict(w2=None), 1),
    (dict(s2=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(x=P + 8), 5), (dict(l=2 * P + 2), 5),
    (dict(w1=3 * P + 4), 5), (dict(s1=4 * P + 1), 5), (dict(w2=6 * P + 8), 5), (dict(s2=7 * P + 1), 5),
    (dict(out=9 * P + 1), 5), (dict(ids=10 * P + 2), 5), (dict(pw=11 * P + 1), 5), (dict(ws=12 * P + 4), 5),
    (dict(size=16), 11), (dict(out=P + 2), 8), (dict(out=3 * P), 8), (dict(out=8 * P), 8), (dict(ids=9 * P), 8),
    (dict(ids=11 * P + 20), 8), (dict(pw=2 * P + 44), 8), (dict(ws=9 * P), 8), (dict(ws=7 * P), 8),
])
def test_moe_refusals(args, status):
    _status(_moe, args, status)


def test_moe_workspace_sizes():
    need = mnb.mnb_moe_workspace(3, 64, 96, 4, 2)
    assert need > 0
    _status(_moe, dict(size=need - 1), 11)
    for bad in ((65, 64, 96, 4, 2), (3, 63, 96, 4, 2), (3, 64, 0, 4, 2), (3, 64, 96, 0, 1), (3, 64, 96, 4, 5),
                (0, 64, 96, 4, 2)):
        assert mnb.mnb_moe_workspace(*bad) == 0


def test_empty_calls():
    c0 = mnb.mnb_counters_get()
    assert _quantize(m=0, A=None, q=None, s=None) == 0
    assert _int8(m=0, A=None, sa=None, B=None, sb=None, out=None) == 0
    assert _int8(N=0, out=None, B=None, sb=None) == 0
    assert _moe(T=0, x=None, out=None, ws=None) == 0
    c1 = mnb.mnb_counters_get()
    assert c1["calls"] == c0["calls"] + 4 and c1["launches"] == c0["launches"]


def test_binding_refuses_cpu_tensors_and_shapes():
    import torch
    A = torch.zeros(2, 64, dtype=torch.float16)
    q = torch.zeros(2, 64, dtype=torch.int8)
    s = torch.zeros(2)
    with pytest.raises(ValueError):
        mnb.quantize_rows_int8(A, q, s)                   # not on the GPU
    with pytest.raises(ValueError):
        mnb.quantize_rows_int8(A[0], q, s)                # not 2-D
    with pytest.raises(ValueError):
        mnb.matmul_int8(A, None, q, s, None, A)
    with pytest.raises(ValueError):
        mnb.matmul_int8(A, None, q[0], s, None, A)
    with pytest.raises(ValueError):
        mnb.moe_nbits(A, A, q, q, None, q, q, None, A, 1)   # weights not 3-D
