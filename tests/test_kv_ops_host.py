"""Refusals, workspace sizes and empty calls of append_kv_int8, attention_int8
and matmul_lora, without a GPU: every check runs on the host before anything is
launched, so the addresses below are never dereferenced."""
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


def _cache(pages=9, size=16, heads=2, D=64, kp=P, vp=2 * P, ks=3 * P, vs=4 * P):
    return mnb.mnb_kv_cache(pages, size, heads, D, kp, vp, ks, vs)


def _batch(S=3, T=5, width=4, starts=5 * P, lengths=6 * P, table=7 * P):
    return mnb.mnb_kv_batch(S, T, width, starts, lengths, table)


def _split(args):
    cache = {k: args.pop(k) for k in list(args) if k in ("pages", "size", "heads", "D", "kp", "vp", "ks", "vs")}
    batch = {k: args.pop(k) for k in list(args) if k in ("S", "T", "width", "starts", "lengths", "table")}
    return _cache(**cache), _batch(**batch)


def _append(null_cache=False, null_batch=False, dtype=mnb.MNB_F16, k=8 * P, k_stride=128, v=9 * P, v_stride=128,
            q=10 * P, q_stride=256, q_out=11 * P, q_out_stride=256, q_heads=4, cos=12 * P, sin=13 * P, rot=64, rows=64,
            **other):
    c, b = _split(other)
    assert not other
    return mnb.lib().append_kv_int8(None if null_cache else ctypes.byref(c), None if null_batch else ctypes.byref(b),
                                    dtype, k, k_stride, v, v_stride, q, q_stride, q_out, q_out_stride, q_heads, cos,
                                    sin, rot, rows, 0, None)


SHARED = [
    (dict(null_cache=True), 1), (dict(null_batch=True), 1), (dict(T=-1), 6), (dict(T=(1 << 20) + 1), 6),
    (dict(pages=-1), 2), (dict(pages=1 << 31), 2), (dict(size=8), 2), (dict(size=48), 2), (dict(size=512), 2),
    (dict(heads=0), 2), (dict(heads=257), 2), (dict(D=32), 2), (dict(D=96), 2), (dict(D=512), 2), (dict(S=-1), 2),
    (dict(S=65537), 2), (dict(width=-1), 2), (dict(width=(1 << 20) + 1), 2), (dict(dtype=mnb.MNB_F32), 4),
    (dict(dtype=mnb.MNB_I8), 4), (dict(dtype=-1), 4), (dict(starts=None), 1), (dict(lengths=None), 1),
    (dict(table=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(ks=None), 1), (dict(vs=None), 1),
    (dict(starts=5 * P + 2), 5), (dict(lengths=6 * P + 1), 5), (dict(table=7 * P + 2), 5), (dict(kp=P + 8), 5),
    (dict(vp=2 * P + 4), 5), (dict(ks=3 * P + 2), 5), (dict(vs=4 * P + 1), 5),
]


@pytest.mark.parametrize("args,status", SHARED + [
    (dict(rot=-16), 2), (dict(rot=8), 2), (dict(rot=80), 2), (dict(rows=63), 2), (dict(q_heads=-1), 2),
    (dict(q_heads=256 * 64 + 1), 2), (dict(k_stride=120), 2), (dict(k_stride=132), 2), (dict(v_stride=64), 2),
    (dict(q_stride=128), 2), (dict(q_out_stride=257), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1),
    (dict(q_out=None), 1), (dict(q_heads=0), 1), (dict(q=None, q_out=None), 1), (dict(cos=None), 1),
    (dict(sin=None), 1), (dict(k=8 * P + 8), 5), (dict(v=9 * P + 2), 5), (dict(q=10 * P + 4), 5),
    (dict(q_out=11 * P + 8), 5), (dict(cos=12 * P + 4), 5), (dict(sin=13 * P + 8), 5),
    # written buffers over inputs and each other
    (dict(kp=8 * P), 8), (dict(vp=9 * P + 64), 8), (dict(ks=5 * P), 8), (dict(vs=7 * P + 40), 8), (dict(kp=12 * P), 8),
    (dict(vp=P + 1024), 8), (dict(ks=2 * P), 8), (dict(vs=3 * P + 4), 8), (dict(q_out=8 * P), 8),
    (dict(q_out=9 * P + 512), 8), (dict(q_out=13 * P), 8), (dict(q_out=P), 8), (dict(q_out=6 * P), 8),
    (dict(q_out=10 * P + 16), 8), (dict(q_out=10 * P, q_out_stride=264), 8),
    # parts of one buffer whose rows meet: q_out's last head is k's first
    (dict(q_out=8 * P - 384, k_stride=512, q_out_stride=512), 8),
])
def test_append_refusals(args, status):
    _status(_append, dict(args), status)


def test_append_takes_parts_of_one_buffer():
    """q, k, v and q_out between each other with one stride pass the checks (and
    end at the launch: there is no GPU here, or they are empty)."""
    fused = dict(q=8 * P, k=8 * P + 512, v=8 * P + 768, q_stride=512, k_stride=512, v_stride=512)
    for q_out, stride in ((8 * P, 512), (9 * P, 256), (8 * P + 1024 - 512 + 512, 512)):
        args = dict(fused, q_out=q_out, q_out_stride=stride)
        if q_out == 8 * P + 1024:          # the next row's q
            _status(_append, args, 8)
        else:
            assert _append(S=0, **args) == 0


def _attention(null_cache=False, null_batch=False, dtype=mnb.MNB_F16, q=8 * P, q_stride=256, q_heads=4, scale=0.125,
               out=9 * P, out_stride=256, most=0, ws=10 * P, room=1 << 30, **other):
    c, b = _split(other)
    assert not other
    return mnb.lib().attention_int8(None if null_cache else ctypes.byref(c), None if null_batch else ctypes.byref(b),
                                    dtype, q, q_stride, q_heads, scale, out, out_stride, most, ws, room, None)


@pytest.mark.parametrize("args,status", SHARED + [
    (dict(q_heads=0), 2), (dict(q_heads=5), 2), (dict(q_heads=130), 2), (dict(q_stride=192), 2), (dict(q_stride=260), 2),
    (dict(out_stride=255), 2), (dict(most=-1), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2),
    (dict(q=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(q=8 * P + 8), 5), (dict(out=9 * P + 4), 5),
    (dict(ws=10 * P + 8), 5), (dict(room=1000), 11), (dict(out=8 * P), 8), (dict(out=8 * P + 256), 8), (dict(out=P), 8),
    (dict(out=4 * P), 8), (dict(out=7 * P), 8), (dict(ws=8 * P), 8), (dict(ws=9 * P), 8), (dict(ws=2 * P), 8),
    (dict(ws=6 * P), 8),
])
def test_attention_refusals(args, status):
    _status(_attention, dict(args), status)


def test_attention_workspace():
    need = mnb.mnb_attention_workspace(5, 3, 4, 2, 64)
    assert need > 0
    _status(_attention, dict(room=need - 1), 11)
    for bad in ((-1, 3, 4, 2, 64), ((1 << 20) + 1, 3, 4, 2, 64), (0, 3, 4, 2, 64), (5, 0, 4, 2, 64), (5, -1, 4, 2, 64),
                (5, 3, 3, 2, 64), (5, 3, 4, 0, 64), (5, 3, 4, 2, 80), (5, 3, 130, 2, 64)):
        assert mnb.mnb_attention_workspace(*bad) == 0


def _lora(x=P, xd=mnb.MNB_F16, x_stride=64, m=3, K=64, N=40, R=8, n=2, ids=2 * P, A=3 * P, B=4 * P, scaling=5 * P,
          base=6 * P, base_stride=40, out=7 * P, out_stride=40, od=mnb.MNB_F16, ws=8 * P, size=1 << 24):
    return mnb.lib().matmul_lora(x, xd, x_stride, m, K, N, R, n, ids, A, B, scaling, base, base_stride, out, out_stride,
                                 od, ws, size, None)


@pytest.mark.parametrize("args,status", [
    (dict(m=-1), 6), (dict(m=(1 << 20) + 1), 6), (dict(K=-16), 2), (dict(K=24), 2), (dict(K=(1 << 24) + 16), 2),
    (dict(N=-1), 2), (dict(N=mnb.MNB_MAX_N_INT8 + 1), 2), (dict(R=0), 2), (dict(R=12), 2), (dict(R=264), 2),
    (dict(n=-1), 2), (dict(n=65537), 2), (dict(x_stride=48), 2), (dict(x_stride=68), 2), (dict(out_stride=39), 2),
    (dict(base_stride=8), 2), (dict(xd=mnb.MNB_I8), 4), (dict(xd=mnb.MNB_F32), 4), (dict(od=mnb.MNB_F32), 4),
    (dict(x=None), 1), (dict(ids=None), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(K=0, A=None, x=None, B=None), 1), (dict(x=P + 8), 5), (dict(ids=2 * P + 2), 5), (dict(A=3 * P + 8), 5),
    (dict(B=4 * P + 4), 5), (dict(scaling=5 * P + 2), 5), (dict(base=6 * P + 1), 5), (dict(out=7 * P + 1), 5),
    (dict(ws=8 * P + 8), 5), (dict(size=8), 11), (dict(out=P), 8), (dict(out=2 * P), 8), (dict(out=3 * P + 64), 8),
    (dict(out=4 * P), 8), (dict(out=5 * P), 8), (dict(out=6 * P + 2), 8), (dict(out=6 * P, out_stride=48), 8),
    (dict(ws=P), 8), (dict(ws=6 * P), 8), (dict(ws=7 * P), 8), (dict(ws=3 * P), 8),
])
def test_lora_refusals(args, status):
    _status(_lora, dict(args), status)


def test_lora_workspace():
    need = mnb.mnb_lora_workspace(300, 4096, 4096, 32, 5)
    assert need >= 300 * 32 * 4
    _status(_lora, dict(m=300, K=4096, x_stride=4096, N=4096, base_stride=4096, out_stride=4096, R=32, n=5, size=need - 1), 11)
    for bad in ((-1, 64, 40, 8, 2), (3, 65, 40, 8, 2), (3, 64, -1, 8, 2), (3, 64, 40, 4, 2), (3, 64, 40, 8, -1),
                (0, 64, 40, 8, 2), (3, 64, 0, 8, 2)):
        assert mnb.mnb_lora_workspace(*bad) == 0


def test_empty_calls():
    c0 = mnb.mnb_counters_get()
    assert _append(T=0, k=None, v=None, q=None, q_out=None, q_heads=0, kp=None, starts=None) == 0
    assert _append(S=0) == 0 and _append(width=0, rows=0) == 0
    assert _attention(T=0, q=None, out=None, ws=None, kp=None) == 0
    assert _attention(S=0, q=None) == 0
    assert _lora(m=0, x=None, ids=None, out=None) == 0
    assert _lora(N=0, out=None, B=None, out_stride=0, base_stride=0) == 0
    c1 = mnb.mnb_counters_get()
    assert c1["calls"] == c0["calls"] + 7 and c1["launches"] == c0["launches"]


def test_binding_refuses_cpu_tensors_and_shapes():
    import torch
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    k = torch.zeros(3, 4, 16, 64, dtype=torch.int8)
    s = torch.zeros(3, 4)
    with pytest.raises(ValueError):
        mnb.append_kv_int8(x, x, None, None, i, i[:1], i[None], k, k.mT.contiguous(), s, s)    # not on the GPU
    with pytest.raises(ValueError):
        mnb.append_kv_int8(x[0], x, None, None, i, i[:1], i[None], k, k, s, s)                 # not 3-D
    with pytest.raises(ValueError):
        mnb.attention_int8(x, i, i[:1], i[None], k, k, s, s, x)
    with pytest.raises(ValueError):
        mnb.attention_int8(x[:, 0], i, i[:1], i[None], k, k, s, s, x)
    with pytest.raises(ValueError):
        mnb.matmul_lora(x[0], i, x, x, None, x[0])
    with pytest.raises(ValueError):
        mnb.matmul_lora(x, i, x, x, None, x[0])


def test_module_refuses_what_is_no_gpu_tensor():
    """The compiled part of the binding on CPU tensors and other objects: errors in
    Python's manner, nothing launched."""
    import torch
    N = mnb._load_native()
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    k = torch.zeros(3, 4, 16, 64, dtype=torch.int8)
    s = torch.zeros(3, 4)
    cache = (i, i[:2], i[None], k, k, s, s)
    c0 = mnb.mnb_counters_get()
    for call, error in ((lambda: N.append_kv_int8(x), TypeError), (lambda: N.attention_int8(), TypeError),
                        (lambda: N.matmul_lora(1, 2, 3, 4, 5, 6, 7, 8, 9), TypeError),
                        (lambda: N.append_kv_int8(x, x, None, None, *cache, None, None, False, 0), ValueError),
                        (lambda: N.append_kv_int8(x[0], x, None, None, *cache, None, None, False, 0), ValueError),
                        (lambda: N.append_kv_int8(x.float(), x, None, None, *cache, None, None, False, 0), TypeError),
                        (lambda: N.append_kv_int8(x, None, None, None, *cache, None, None, False, 0), ValueError),
                        (lambda: N.attention_int8(x, *cache, x, None, None, None, 0), ValueError),
                        (lambda: N.attention_int8("x", *cache, x, None, None, None, 0), TypeError),
                        (lambda: N.matmul_lora(x[0], i, x, x, None, x[0], None, None, 0), ValueError)):
        with pytest.raises(error):
            call()
    assert mnb.mnb_counters_get() == c0
