"""The cache, attention and adapter calls as programs make them: the attention
half of a served layer, eager and captured; refusals of tensors; raw streams;
several host threads at once."""
import threading

import pytest
import torch

import block_wise_int4_matmulnbits_amd as mnb
from tests import gpu_util as G
from tests import kv_ref as R
from tests import test_gpu_int8 as I8
from tests import test_gpu_moe as MOE

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


class Layer:
    """4-bit projection to queries, keys and values with adapters beside it, the
    cache, attention, 8-bit projection back with adapters beside it."""

    def __init__(self, H, hq, heads, D, rank, n, seed):
        g = torch.Generator().manual_seed(seed)
        self.H, self.hq, self.heads, self.D = H, hq, heads, D
        self.W = (hq + 2 * heads) * D
        B, S, Z = MOE._matrix(g, 1, self.W, H, True, 5e-4, 4e-3)
        self.qkv = (B[0].cuda(), S[0].cuda(), Z[0].cuda())
        self.A1 = (torch.randn(n, rank, H, generator=g) * H ** -0.5).to(F16).cuda()
        self.B1 = (torch.randn(n, self.W, rank, generator=g) * 0.3).to(F16).cuda()
        self.o = torch.randint(-127, 128, (H, hq * D), generator=g, dtype=torch.int8).cuda()
        self.o_scales = (torch.rand(H, generator=g) * 2e-4 + 1e-5).cuda()
        self.A2 = (torch.randn(n, rank, hq * D, generator=g) * (hq * D) ** -0.5).to(F16).cuda()
        self.B2 = (torch.randn(n, H, rank, generator=g) * 0.3).to(F16).cuda()
        self.scaling = (torch.rand(n, generator=g) + 0.5).cuda()
        angle = torch.rand(512, D // 2, generator=g, dtype=torch.float64) * 6.2
        self.cos, self.sin = angle.cos().float().cuda(), angle.sin().float().cuda()

    def step(self, x, ids, b, bufs):
        """b: (starts, lengths, table, k_pages, v_pages, k_scales, v_scales)."""
        T = x.shape[0]
        mnb.matmul_nbits(x, *self.qkv, bufs["p"])
        mnb.matmul_lora(x, ids, self.A1, self.B1, bufs["p"], bufs["qkv"], scaling=self.scaling)
        qkv = bufs["qkv"].view(T, self.hq + 2 * self.heads, self.D)
        q, k, v = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.heads], qkv[:, self.hq + self.heads:]
        mnb.append_kv_int8(k, v, self.cos, self.sin, *b, q=q, q_out=bufs["q"])
        mnb.attention_int8(bufs["q"], *b, bufs["a"])
        flat = bufs["a"].view(T, self.hq * self.D)
        mnb.matmul_int8(flat, None, self.o, self.o_scales, None, bufs["o"])
        mnb.matmul_lora(flat, ids, self.A2, self.B2, bufs["o"], bufs["o"], scaling=self.scaling)

    def buffers(self, T):
        e = lambda *shape: torch.full(shape, 3.0, dtype=F16, device="cuda")
        return {"p": e(T, self.W), "qkv": e(T, self.W), "q": e(T, self.hq, self.D), "a": e(T, self.hq, self.D),
                "o": e(T, self.H)}


@pytest.mark.parametrize("new,before", [([1], [100]), ([1, 1, 1, 1], [0, 3, 64, 200]), ([2, 70, 1, 9], [30, 0, 128, 55])],
                         ids=["token", "tokens", "mixed"])
def test_layer_as_served(new, before):
    G.require_gpu()
    L = Layer(512, 8, 2, 64, 16, 3, 7)
    T = sum(new)
    steps = []
    for i in range(3):
        g = torch.Generator().manual_seed(i)
        b = R.Batch(new, [c + i for c in before], 32, 2, 64, seed=i, width=16, spare=4)
        pages = 40
        for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
            t = getattr(b, name)
            setattr(b, name, torch.cat((t, t.new_zeros((pages - t.shape[0],) + t.shape[1:]))))
        b.pages = pages
        x = torch.randn(T, 512, generator=g).to(F16)
        ids = torch.randint(-1, 3, (T,), generator=g).to(torch.int32)
        steps.append((b, x, ids))
    eager = []
    for b, x, ids in steps:
        dev, bufs = b.cuda(), L.buffers(T)
        L.step(x.cuda(), ids.cuda(), dev, bufs)
        torch.cuda.synchronize()
        h = {n: t.cpu() for n, t in bufs.items()}
        eager.append((h, [t.cpu() for t in dev]))
        # Each operator against its formula in 64 bits on the inputs that it got.
        cpu = lambda *ts: [t.cpu() for t in ts]
        want, tol = R.lora(x, ids, *cpu(L.A1, L.B1, L.scaling), h["p"])
        R.check_rows(h["qkv"], want, tol, F16)
        qkv = h["qkv"].view(T, 12, 64)
        want = R.append(b, qkv[:, 8:10], qkv[:, 10:], *cpu(L.cos, L.sin), qkv[:, :8])
        for got, ref in zip(dev[3:], b.cache()):
            assert torch.equal(got.cpu(), ref)
        R.check_rows(h["q"], want, torch.zeros_like(want), F16)
        want, tol = R.attention(b, h["q"], 64 ** -0.5)
        R.check_rows(h["a"], want, tol, F16)
        proj = torch.empty(T, 512, dtype=F16, device="cuda")
        mnb.matmul_int8(bufs["a"].view(T, 512), None, L.o, L.o_scales, None, proj)
        want, tol = R.lora(h["a"].view(T, 512), ids, *cpu(L.A2, L.B2, L.scaling), proj.cpu())
        R.check_rows(h["o"], want, tol, F16)
    # A captured step with other tokens, lengths, pages and adapters, eager work between.
    fresh = R.Batch(new, before, 32, 2, 64, seed=0, width=16, spare=4)
    del fresh
    first = steps[0]
    dev = [t.clone() for t in first[0].cuda()]
    x, ids, bufs = first[1].cuda(), first[2].cuda(), L.buffers(T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step(x, ids, dev, bufs)
    for i in (1, 2, 0, 1):
        # the reference left b's cache as after the step: storing the same tokens again changes nothing
        for dst, src in zip(dev, steps[i][0].cuda()):
            dst.copy_(src)
        x.copy_(steps[i][1])
        ids.copy_(steps[i][2])
        graph.replay()
        torch.cuda.synchronize()
        for n, t in bufs.items():
            assert torch.equal(t.cpu(), eager[i][0][n]), n
        for got, ref in zip(dev[3:], eager[i][1][3:]):
            assert torch.equal(got.cpu(), ref)
        L.step(x, ids, [t.clone() for t in dev], L.buffers(T))
        torch.cuda.synchronize()


@pytest.mark.parametrize("new,before", [([1], [100]), ([1, 1, 1, 1], [0, 3, 64, 200]), ([2, 70, 1, 9], [30, 0, 128, 55])],
                         ids=["token", "tokens", "mixed"])
def test_captured_layer_from_the_cache_before(new, before):
    """A captured step replayed over caches as they are before it: what it has to
    store is not there yet, and the eager step's cache and outputs are."""
    G.require_gpu()
    L = Layer(512, 8, 2, 64, 16, 3, 11)
    T = sum(new)
    steps = []
    for i in range(3):
        g = torch.Generator().manual_seed(10 + i)
        b = R.Batch(new, [c + i for c in before], 32, 2, 64, seed=i, width=16, spare=4)
        pages = 40
        for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
            t = getattr(b, name)
            setattr(b, name, torch.cat((t, t.new_zeros((pages - t.shape[0],) + t.shape[1:]))))
        b.pages = pages
        x, ids = torch.randn(T, 512, generator=g).to(F16).cuda(), torch.randint(-1, 3, (T,), generator=g).to(torch.int32).cuda()
        cache, bufs = b.cuda(), L.buffers(T)
        clean = [t.clone() for t in cache]
        L.step(x, ids, cache, bufs)
        torch.cuda.synchronize()
        for t, was in zip(cache[3:5], clean[3:5]):
            assert not torch.equal(t, was)
        steps.append((x, ids, clean, cache, bufs))
    x, ids, dev = steps[0][0].clone(), steps[0][1].clone(), [t.clone() for t in steps[0][2]]
    bufs = L.buffers(T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step(x, ids, dev, bufs)
    for i in (1, 2, 0, 1):
        sx, sids, clean, after, want = steps[i]
        for dst, src in zip([x, ids] + dev, [sx, sids] + clean):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(dev[3:], after[3:]):
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
        for n, t in bufs.items():
            assert torch.equal(t, want[n]), n
        L.step(x, ids, [t.clone() for t in clean], L.buffers(T))       # eager work between the replays
        torch.cuda.synchronize()


def _calls(seed):
    """Calls of the three operators on inputs of their own: (call(out, stream), shape)."""
    b = R.Batch([1, 40, 2], [300, 20, 77], 16, 2, 64, seed=seed)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(b.T, 8, 64, generator=g).to(F16).cuda()
    args = b.cuda()
    x = torch.randn(50, 256, generator=g).to(F16).cuda()
    ids = torch.randint(-1, 4, (50,), generator=g).to(torch.int32).cuda()
    A = torch.randn(4, 16, 256, generator=g).to(F16).cuda()
    B = torch.randn(4, 300, 16, generator=g).to(F16).cuda()
    k = torch.randn(b.T, 2, 64, generator=g).to(F16).cuda()
    cache = [t.clone() for t in args]
    cos = torch.ones(b.width * 16, 32, device="cuda")

    def attention(out, stream=None):
        return mnb.attention_int8(q, *args, out, stream=stream)

    def lora(out, stream=None):
        return mnb.matmul_lora(x, ids, A, B, None, out, stream=stream)

    def append(out, stream=None):
        return mnb.append_kv_int8(k, k, cos, cos, *cache, q=q, q_out=out, stream=stream)

    return [(attention, (b.T, 8, 64)), (lora, (50, 300)), (append, (b.T, 8, 64))]


def test_raw_stream_handles():
    G.require_gpu()
    side = torch.cuda.Stream()
    for call, shape in _calls(3):
        want = call(torch.empty(shape, dtype=F16, device="cuda"))
        torch.cuda.synchronize()
        for stream in (side, side.cuda_stream, 0):
            out = torch.full(shape, float("nan"), dtype=F16, device="cuda")
            torch.cuda.synchronize()
            for _ in range(3):
                assert call(out, stream) is out
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_threads():
    """Each thread on a stream of its own, its calls back to back; a workspace
    shared between them would show."""
    G.require_gpu()
    calls = _calls(1) + _calls(2)
    want = [call(torch.empty(shape, dtype=F16, device="cuda")) for call, shape in calls]
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


def test_refusals_of_tensors():
    """Shapes, types, strides and places that the binding refuses, and what the
    library refuses through it; nothing is launched."""
    G.require_gpu()
    b = R.Batch([3], [20], 16, 2, 64, seed=1)
    c = b.cuda()
    q = torch.zeros(3, 4, 64, dtype=F16, device="cuda")
    k = torch.zeros(3, 2, 64, dtype=F16, device="cuda")
    out = torch.empty_like(q)
    cos = torch.ones(b.width * 16, 32, device="cuda")
    x = torch.zeros(5, 64, dtype=F16, device="cuda")
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    A, B = torch.zeros(2, 8, 64, dtype=F16, device="cuda"), torch.zeros(2, 30, 8, dtype=F16, device="cuda")
    y = torch.zeros(5, 30, dtype=F16, device="cuda")

    def swap(i, t):
        return c[:i] + [t] + c[i + 1:]

    att = lambda q=q, c=c, out=out, **kw: mnb.attention_int8(q, *c, out, **kw)
    app = lambda k=k, v=k, cos=cos, sin=cos, c=c, **kw: mnb.append_kv_int8(k, v, cos, sin, *c, **kw)
    lor = lambda x=x, ids=ids, A=A, B=B, base=y, out=y, **kw: mnb.matmul_lora(x, ids, A, B, base, out, **kw)
    V, T, M = ValueError, TypeError, mnb.MnbError
    cases = [
        (V, lambda: att(q=q.cpu())), (T, lambda: att(q=q.float())), (V, lambda: att(q=q[0])),
        (V, lambda: att(q=q.transpose(0, 1))), (V, lambda: att(q=q[..., ::2])), (T, lambda: att(out=out.to(BF16))),
        (V, lambda: att(out=out[:2])), (V, lambda: att(out=out.cpu())), (V, lambda: att(c=swap(0, c[0][:1]))),
        (T, lambda: att(c=swap(0, c[0].long()))), (V, lambda: att(c=swap(1, c[1].cpu()))), (V, lambda: att(c=swap(2, c[2][0]))),
        (V, lambda: att(c=swap(4, c[4].transpose(2, 3)))), (T, lambda: att(c=swap(3, c[3].view(torch.uint8)))),
        (V, lambda: att(c=swap(5, c[5][:1]))), (T, lambda: att(c=swap(6, c[6].double()))),
        (V, lambda: att(workspace=torch.empty(10 ** 8, dtype=torch.uint8))), (M, lambda: att(out=q)),
        (M, lambda: att(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))), (M, lambda: att(scale=float("nan"))),
        (M, lambda: att(max_tokens=-1)), (M, lambda: att(q=q[:, :3], out=out[:, :3])),
        (T, lambda: app(k=k.double())), (V, lambda: app(k=k[:, :1], v=k[:, :1])), (V, lambda: app(v=k[:2])),
        (V, lambda: app(sin=None)), (V, lambda: app(cos=None)), (V, lambda: app(q=q)), (V, lambda: app(q_out=q)),
        (T, lambda: app(cos=cos.half(), sin=cos.half())), (V, lambda: app(sin=cos[:-1])), (M, lambda: app(cos=cos[:-1], sin=cos[:-1])),
        (M, lambda: app(cos=cos[:, :20].contiguous(), sin=cos[:, :20].contiguous())), (V, lambda: app(cos=cos[0], sin=cos[0])),
        (T, lambda: app(q=q.to(BF16), q_out=out.to(BF16))), (V, lambda: app(q=q, q_out=out[:, :2])), (M, lambda: app(q=k, q_out=k)),
        (V, lambda: lor(x=x.cpu())), (T, lambda: lor(A=A.to(BF16))), (V, lambda: lor(B=B[:1])), (V, lambda: lor(A=A[:, :, ::2])),
        (T, lambda: lor(ids=ids.long())), (V, lambda: lor(ids=ids[:3])), (V, lambda: lor(x=x.t())), (T, lambda: lor(base=y.to(BF16))),
        (V, lambda: lor(base=y[:, :10])), (M, lambda: lor(x=x[:, :24], A=A[:, :, :24].contiguous())),
        (T, lambda: lor(scaling=torch.ones(2, dtype=F16, device="cuda"))), (V, lambda: lor(scaling=torch.ones(3, device="cuda"))),
        (M, lambda: lor(base=None, out=x[:, :30])),
    ]
    c0 = mnb.mnb_counters_get()
    for i, (error, call) in enumerate(cases):
        with pytest.raises(error):
            call()
            print("case %d was taken" % i)
    assert mnb.mnb_counters_get() == c0
    torch.cuda.synchronize()
