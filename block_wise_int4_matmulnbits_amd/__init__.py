"""Python binding of libmnb, the block-wise INT4 MatMulNBits products, 8-bit
products and 4-bit expert layers for MI355X (gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libmnb.so`` (built in-tree by ``build.py``).  Functions carry the
names of the C entry points declared in ``include/mnb.h``.  torch supplies
device memory and streams; nothing here computes on the host, and there is
no fallback: if the library is missing, importing the entry points raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmnb.so")

MNB_F16 = 0
MNB_BF16 = 1
MNB_F32 = 2              # router logits of moe_nbits
MNB_I8 = 3               # quantised rows of matmul_int8
MNB_MAX_M = 8            # decode kernels; prefill up to MNB_MAX_ROWS
MNB_MAX_ROWS = 1 << 20
MNB_MAX_SPLIT_WORKSPACE = 32 << 20   # bytes of K-split partial sums a default plan may take
MNB_MAX_K_INT8 = 131056
MNB_MAX_N_INT8 = 2147483136
MNB_MOE_MAX_TOKENS = 64
MNB_MOE_MAX_EXPERTS = 512
MNB_MOE_MAX_TOP_K = 16
MNB_MOE_MAX_WIDTH = 65536
MNB_LAYOUT_NATURAL = 0   # stored weight layouts (mnb_repack_weights)
MNB_LAYOUT_EVEN_ODD = 1

STATUS = {
    0: "MNB_OK", 1: "MNB_ERR_NULL", 2: "MNB_ERR_SHAPE", 3: "MNB_ERR_BLOCK",
    4: "MNB_ERR_DTYPE", 5: "MNB_ERR_ALIGN", 6: "MNB_ERR_M_RANGE",
    7: "MNB_ERR_HIP", 8: "MNB_ERR_ALIAS", 9: "MNB_ERR_PLAN", 10: "MNB_ERR_LAYOUT",
    11: "MNB_ERR_WORKSPACE",
}


class MnbError(RuntimeError):
    def __init__(self, status, lib=None):
        self.status = status
        text = lib.mnb_status_string(status).decode() if lib is not None else ""
        name = STATUS.get(status, str(status))
        if status == 7 and lib is not None:
            text += " (hipError_t %d)" % lib.mnb_last_hip_error()
        super().__init__("%s: %s" % (name, text))


class mnb_plan(ctypes.Structure):
    _fields_ = [("engine", ctypes.c_int32),
                ("lanes_per_col", ctypes.c_int32),
                ("blocks_per_lane", ctypes.c_int32),
                ("cols_per_tile", ctypes.c_int32),
                ("waves_per_wg", ctypes.c_int32),
                ("workgroups", ctypes.c_int32),
                ("interleave", ctypes.c_int32),
                ("threads_per_wg", ctypes.c_int32),
                ("k_chunks", ctypes.c_int32),
                ("row_tiles", ctypes.c_int32),
                ("b_layout", ctypes.c_int32),
                ("k_splits", ctypes.c_int32),
                ("a_via_lds", ctypes.c_int32)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class mnb_counters(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_uint64),
                ("launches", ctypes.c_uint64),
                ("elements_f16", ctypes.c_uint64),
                ("elements_bf16_direct", ctypes.c_uint64),
                ("row_batched_launches", ctypes.c_uint64)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class mnb_kernel_info(ctypes.Structure):
    _fields_ = [("vgprs", ctypes.c_int32), ("sgprs", ctypes.c_int32),
                ("lds_bytes", ctypes.c_int32), ("max_threads", ctypes.c_int32),
                ("wgs_per_cu", ctypes.c_int32)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class mnb_moe_weights(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int64), ("hidden", ctypes.c_int64), ("inter", ctypes.c_int64),
                ("gate_up", ctypes.c_void_p), ("gate_up_scales", ctypes.c_void_p),
                ("gate_up_zero_points", ctypes.c_void_p),
                ("down", ctypes.c_void_p), ("down_scales", ctypes.c_void_p),
                ("down_zero_points", ctypes.c_void_p), ("block", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None

EXPORTS = ("matmul_nbits", "matmul_nbits_planned", "matmul_nbits_noalloc", "mnb_plan_default",
           "mnb_plan_check", "mnb_counters_get", "mnb_counters_reset",
           "mnb_get_kernel_info", "mnb_status_string", "mnb_last_hip_error",
           "mnb_abi_version", "mnb_repack_weights", "quantize_rows_int8", "matmul_int8",
           "mnb_int8_workspace", "moe_nbits", "mnb_moe_workspace")


def lib():
    """Load libmnb.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                "libmnb.so is not built (%s); run __graft_entry__.build() or "
                "python block_wise_int4_matmulnbits_amd/build.py" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.matmul_nbits.restype = i32
        L.matmul_nbits.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, i32, vp,
                                   i32, vp]
        L.matmul_nbits_planned.restype = i32
        L.matmul_nbits_planned.argtypes = L.matmul_nbits.argtypes + [
            ctypes.POINTER(mnb_plan)]
        L.matmul_nbits_noalloc.restype = i32
        L.matmul_nbits_noalloc.argtypes = L.matmul_nbits.argtypes
        L.mnb_plan_default.restype = i32
        L.mnb_plan_default.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(mnb_plan)]
        L.mnb_plan_check.restype = i32
        L.mnb_plan_check.argtypes = [i64, i64, i64, ctypes.POINTER(mnb_plan)]
        L.mnb_counters_get.restype = None
        L.mnb_counters_get.argtypes = [ctypes.POINTER(mnb_counters)]
        L.mnb_counters_reset.restype = None
        L.mnb_counters_reset.argtypes = []
        L.mnb_get_kernel_info.restype = i32
        L.mnb_get_kernel_info.argtypes = [i64, i64, ctypes.POINTER(mnb_plan),
                                          ctypes.POINTER(mnb_kernel_info)]
        L.mnb_status_string.restype = ctypes.c_char_p
        L.mnb_status_string.argtypes = [i32]
        L.mnb_last_hip_error.restype = i32
        L.mnb_last_hip_error.argtypes = []
        L.mnb_abi_version.restype = i32
        L.mnb_abi_version.argtypes = []
        L.mnb_repack_weights.restype = i32
        L.mnb_repack_weights.argtypes = [vp, i32, vp, i32, i64, i64, vp]
        L.quantize_rows_int8.restype = i32
        L.quantize_rows_int8.argtypes = [vp, i32, i64, i64, vp, vp, vp]
        L.matmul_int8.restype = i32
        L.matmul_int8.argtypes = [vp, i32, vp, i64, i64, i64, vp, vp, vp, vp, i32, vp,
                                  ctypes.c_size_t, vp]
        L.mnb_int8_workspace.restype = ctypes.c_size_t
        L.mnb_int8_workspace.argtypes = [i32, i64, i64, i64]
        L.moe_nbits.restype = i32
        L.moe_nbits.argtypes = [vp, i32, i64, vp, i32, i32, i32, ctypes.POINTER(mnb_moe_weights),
                                vp, i32, vp, vp, vp, ctypes.c_size_t, vp]
        L.mnb_moe_workspace.restype = ctypes.c_size_t
        L.mnb_moe_workspace.argtypes = [i64, i64, i64, i64, i32]
        _lib = L
        return L


# ---------------------------------------------------------------- marshalling
def _dtype_code(t):
    import torch
    if t.dtype == torch.float16:
        return MNB_F16
    if t.dtype == torch.bfloat16:
        return MNB_BF16
    raise TypeError("expected float16 or bfloat16, got %s" % t.dtype)


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status, L):
    if status != 0:
        raise MnbError(status, L)


def _tensor_args(A, Bpacked, scales, zero_points, out):
    if A.dim() != 2 or out.dim() != 2 or Bpacked.dim() != 2 or scales.dim() != 2:
        raise ValueError("A, Bpacked, scales and out must be 2-D")
    m, K = A.shape
    N = Bpacked.shape[0]
    for name, t in (("A", A), ("Bpacked", Bpacked), ("scales", scales), ("out", out)):
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    if zero_points is not None and not zero_points.is_contiguous():
        raise ValueError("zero_points must be contiguous")
    if tuple(out.shape) != (m, N):
        raise ValueError("out must be [m, N] = [%d, %d]" % (m, N))
    if tuple(Bpacked.shape) != (N, K // 2) or Bpacked.element_size() != 1:
        raise ValueError("Bpacked must be uint8 [N, K/2]")
    if tuple(scales.shape) != (N, K // 32) or scales.element_size() != 2:
        raise ValueError("scales must be 16-bit [N, K/32] (fp16 bit patterns)")
    if zero_points is not None and (tuple(zero_points.shape) != (N, (K // 32 + 1) // 2)
                                    or zero_points.element_size() != 1):
        raise ValueError("zero_points must be uint8 [N, ceil(K/64)]")
    return (A.data_ptr(), _dtype_code(A), m, K, N, Bpacked.data_ptr(),
            scales.data_ptr(),
            zero_points.data_ptr() if zero_points is not None else None,
            out.data_ptr(), _dtype_code(out))


def matmul_nbits(A, Bpacked, scales, zero_points, out, block=32, stream=None):
    """out[m, N] = A[m, K] @ dequant(Bpacked, scales, zero_points)^T on the GPU.

    A: fp16/bf16 [m, K]; Bpacked: uint8 [N, K/2]; scales: fp16 [N, K/32];
    zero_points: uint8 [N, ceil(K/64)] or None (zero point 8);
    out: fp16/bf16 [m, N], fully overwritten.  Queued on ``stream``
    (default: torch's current stream on A's device); returns ``out``.
    """
    L = lib()
    a_ptr, a_dt, m, K, N, b_ptr, s_ptr, z_ptr, o_ptr, o_dt = _tensor_args(
        A, Bpacked, scales, zero_points, out)
    st = L.matmul_nbits(a_ptr, a_dt, m, K, N, b_ptr, s_ptr, z_ptr, block, o_ptr,
                        o_dt, _stream_handle(stream, A.device))
    _check(st, L)
    return out


def matmul_nbits_noalloc(A, Bpacked, scales, zero_points, out, block=32, stream=None):
    """matmul_nbits that allocates no device memory: a split plan's partial
    sums go to the library's fixed per-device workspace (calls that overlap
    on one device race)."""
    L = lib()
    a_ptr, a_dt, m, K, N, b_ptr, s_ptr, z_ptr, o_ptr, o_dt = _tensor_args(
        A, Bpacked, scales, zero_points, out)
    st = L.matmul_nbits_noalloc(a_ptr, a_dt, m, K, N, b_ptr, s_ptr, z_ptr, block, o_ptr,
                                o_dt, _stream_handle(stream, A.device))
    _check(st, L)
    return out


def matmul_nbits_planned(A, Bpacked, scales, zero_points, out, plan, block=32,
                         stream=None):
    """matmul_nbits with an explicit ``mnb_plan`` (or dict of its fields)."""
    L = lib()
    if isinstance(plan, dict):
        plan = mnb_plan(**{k: v for k, v in plan.items()
                           if k in dict(mnb_plan._fields_)})
    a_ptr, a_dt, m, K, N, b_ptr, s_ptr, z_ptr, o_ptr, o_dt = _tensor_args(
        A, Bpacked, scales, zero_points, out)
    st = L.matmul_nbits_planned(a_ptr, a_dt, m, K, N, b_ptr, s_ptr, z_ptr, block,
                                o_ptr, o_dt, _stream_handle(stream, A.device),
                                ctypes.byref(plan))
    _check(st, L)
    return out


def matmul_nbits_raw(A_ptr, a_dtype, m, K, N, B_ptr, scales_ptr, zp_ptr, block,
                     out_ptr, out_dtype, stream=0):
    """Direct C call with integer addresses; returns the status code."""
    return lib().matmul_nbits(A_ptr, a_dtype, m, K, N, B_ptr, scales_ptr, zp_ptr,
                              block, out_ptr, out_dtype, stream)


def mnb_repack_weights(src, src_layout, dst, dst_layout, stream=None):
    """Convert packed weights [N, K/2] (uint8, on the GPU) between stored
    layouts (MNB_LAYOUT_*); ``dst`` may be ``src`` (in place).  Queued on
    ``stream``; returns ``dst``."""
    L = lib()
    if src.dim() != 2 or dst.shape != src.shape or src.element_size() != 1 or dst.element_size() != 1:
        raise ValueError("src and dst must be uint8 [N, K/2] of one shape")
    if not (src.is_contiguous() and dst.is_contiguous()):
        raise ValueError("src and dst must be contiguous")
    N, K = src.shape[0], 2 * src.shape[1]
    st = L.mnb_repack_weights(src.data_ptr(), src_layout, dst.data_ptr(), dst_layout, N, K,
                              _stream_handle(stream, src.device))
    _check(st, L)
    return dst


# ------------------------------------------- 8-bit products and expert layers
# These are called once per layer and token, so their checks are kept to a few
# attribute reads per tensor.
def _expect(name, t, shape, dtype, index):
    """t has this shape and type, and is contiguous and on GPU ``index``."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s must be on the GPU of the first argument, got %s" % (name, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _first(name, t, dim):
    """Index of the GPU that t is on; t must be contiguous and of ``dim`` dimensions."""
    if t.dim() != dim:
        raise ValueError("%s must be %d-D" % (name, dim))
    index = t.get_device()
    if index < 0:
        raise ValueError("%s must be on the GPU" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return index


def _workspace(t, need, workspace, stream, index):
    """A tensor for a call's workspace: the caller's, or one of torch's
    allocator on the call's stream (inside a graph capture: of the graph's own
    pool), so that calls on several streams and captured graphs never share
    one.  The allocator hands its memory on only to later work of that
    stream."""
    import torch
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the GPU of the first argument")
        return workspace
    if stream is None:
        return t.new_empty(need, dtype=torch.uint8)
    on = torch.cuda.ExternalStream(stream, device=t.device) if isinstance(stream, int) else stream
    with torch.cuda.stream(on):
        return t.new_empty(need, dtype=torch.uint8)


def _on_device(index, stream, call, *args):
    """call(*args, stream handle) with GPU ``index`` current."""
    import torch
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _on_device(index, stream, call, *args)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        handle = stream if isinstance(stream, int) else stream.cuda_stream
    _check(call(*args, handle), _lib)


def quantize_rows_int8(A, q, scales, stream=None):
    """Rows of A to 8-bit integers with one scale per row: scales[r] =
    max|A[r]| / 127 and q[r] = rint(127 A[r] / max|A[r]|).

    A: fp16/bf16 [m, K], K a multiple of 16; q: int8 [m, K]; scales: fp32 [m].
    Queued on ``stream`` (default: torch's current stream on A's device);
    returns ``(q, scales)``.
    """
    import torch
    L = _lib or lib()
    index = _first("A", A, 2)
    m, K = A.shape
    _expect("q", q, (m, K), torch.int8, index)
    _expect("scales", scales, (m,), torch.float32, index)
    _on_device(index, stream, L.quantize_rows_int8, A.data_ptr(), _dtype_code(A), m, K, q.data_ptr(),
               scales.data_ptr())
    return q, scales


def matmul_int8(A, a_scales, B, b_scales, bias, out, workspace=None, stream=None):
    """out[m, N] = (A_q[m, K] @ B[N, K]^T) * a_scales[m] * b_scales[N] + bias[N].

    A: int8 [m, K] with a_scales fp32 [m], or fp16/bf16 [m, K] with a_scales
    None (quantised in the call by quantize_rows_int8's rule); K a multiple of
    16; B: int8 [N, K]; b_scales: fp32 [N]; bias: fp32 [N] or None; out:
    fp16/bf16 [m, N], fully overwritten.  workspace: a tensor of at least
    mnb_int8_workspace(...) bytes, or None for one of torch's allocator.
    Queued on ``stream``; returns ``out``.
    """
    import torch
    L = _lib or lib()
    index = _first("A", A, 2)
    m, K = A.shape
    if B.dim() != 2:
        raise ValueError("B must be 2-D")
    N = B.shape[0]
    _expect("B", B, (N, K), torch.int8, index)
    _expect("b_scales", b_scales, (N,), torch.float32, index)
    _expect("out", out, (m, N), out.dtype, index)
    o_dt = _dtype_code(out)
    if bias is not None:
        _expect("bias", bias, (N,), torch.float32, index)
    if A.dtype == torch.int8:
        a_dt = MNB_I8
        if a_scales is None:
            raise ValueError("int8 rows need a_scales")
        _expect("a_scales", a_scales, (m,), torch.float32, index)
    else:
        a_dt = _dtype_code(A)
        if a_scales is not None:
            raise ValueError("a_scales must be None with fp16 or bf16 rows")
    need = L.mnb_int8_workspace(a_dt, m, K, N) if workspace is None else 0
    ws = _workspace(A, need, workspace, stream, index) if need or workspace is not None else None
    _on_device(index, stream, L.matmul_int8, A.data_ptr(), a_dt, None if a_scales is None else a_scales.data_ptr(),
               m, K, N, B.data_ptr(), b_scales.data_ptr(), None if bias is None else bias.data_ptr(), out.data_ptr(),
               o_dt, None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size())
    return out


def mnb_int8_workspace(a_dtype, m, K, N):
    """Workspace bytes of matmul_int8 (a_dtype: MNB_I8, MNB_F16 or MNB_BF16)."""
    return lib().mnb_int8_workspace(a_dtype, m, K, N)


def moe_nbits(x, router_logits, gate_up, gate_up_scales, gate_up_zero_points, down, down_scales, down_zero_points,
              out, top_k, renormalize=True, expert_ids=None, expert_weights=None, block=32, workspace=None,
              stream=None):
    """out[T, H] = the weighted sum of each token's top_k experts, Down(silu(Gate x) * Up x).

    x: fp16/bf16 [T, H], T <= MNB_MOE_MAX_TOKENS; router_logits: fp32, fp16 or
    bf16 [T, E]; gate_up: uint8 [E, 2I, H/2] (the gate's rows first) with
    scales fp16 [E, 2I, H/32] and zero points uint8 [E, 2I, ceil(H/64)] or
    None; down: uint8 [E, H, I/2], likewise; out: fp16/bf16 [T, H], fully
    overwritten.  expert_ids: int32 [T, top_k] and expert_weights: fp32
    [T, top_k] receive the routing where given.  workspace: a tensor of at
    least mnb_moe_workspace(...) bytes, or None for one of torch's
    allocator.  Queued on ``stream``; returns ``out``.
    """
    import torch
    L = _lib or lib()
    index = _first("x", x, 2)
    T, H = x.shape
    if router_logits.dim() != 2 or gate_up.dim() != 3 or down.dim() != 3:
        raise ValueError("router_logits must be 2-D, gate_up and down 3-D")
    E, I = gate_up.shape[0], gate_up.shape[1] // 2
    u8, f16 = torch.uint8, torch.float16
    _expect("router_logits", router_logits, (T, E), router_logits.dtype, index)
    _expect("gate_up", gate_up, (E, 2 * I, H // 2), u8, index)
    _expect("gate_up_scales", gate_up_scales, (E, 2 * I, H // 32), f16, index)
    _expect("down", down, (E, H, I // 2), u8, index)
    _expect("down_scales", down_scales, (E, H, I // 32), f16, index)
    _expect("out", out, (T, H), out.dtype, index)
    z1 = z2 = ids = weights = None
    if gate_up_zero_points is not None:
        _expect("gate_up_zero_points", gate_up_zero_points, (E, 2 * I, (H // 32 + 1) // 2), u8, index)
        z1 = gate_up_zero_points.data_ptr()
    if down_zero_points is not None:
        _expect("down_zero_points", down_zero_points, (E, H, (I // 32 + 1) // 2), u8, index)
        z2 = down_zero_points.data_ptr()
    if expert_ids is not None:
        _expect("expert_ids", expert_ids, (T, top_k), torch.int32, index)
        ids = expert_ids.data_ptr()
    if expert_weights is not None:
        _expect("expert_weights", expert_weights, (T, top_k), torch.float32, index)
        weights = expert_weights.data_ptr()
    w = mnb_moe_weights(E, H, I, gate_up.data_ptr(), gate_up_scales.data_ptr(), z1, down.data_ptr(),
                        down_scales.data_ptr(), z2, block)
    x_dt, o_dt = _dtype_code(x), _dtype_code(out)
    l_dt = MNB_F32 if router_logits.dtype == torch.float32 else _dtype_code(router_logits)
    need = L.mnb_moe_workspace(T, H, I, E, top_k) if workspace is None else 0
    ws = _workspace(x, need, workspace, stream, index) if need or workspace is not None else None
    _on_device(index, stream, L.moe_nbits, x.data_ptr(), x_dt, T, router_logits.data_ptr(), l_dt, top_k,
               1 if renormalize else 0, ctypes.byref(w), out.data_ptr(), o_dt, ids, weights,
               None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size())
    return out


def mnb_moe_workspace(tokens, hidden, inter, experts, top_k):
    """Workspace bytes of moe_nbits."""
    return lib().mnb_moe_workspace(tokens, hidden, inter, experts, top_k)


def mnb_plan_default(m, K, N, num_cus, wgs_per_cu=0):
    p = mnb_plan()
    L = lib()
    _check(L.mnb_plan_default(m, K, N, num_cus, wgs_per_cu, ctypes.byref(p)), L)
    return p


def plan_for_device(m, K, N, num_cus):
    """The plan matmul_nbits picks on the current device: the default plan,
    re-planned with the measured occupancy of the variant it selects."""
    p = mnb_plan_default(m, K, N, num_cus)
    occ = mnb_get_kernel_info(m, K, p)["wgs_per_cu"]
    return mnb_plan_default(m, K, N, num_cus, occ) if occ > 0 else p


def mnb_plan_check(m, K, N, plan):
    """Returns the status code; fills the derived fields of ``plan``."""
    return lib().mnb_plan_check(m, K, N, ctypes.byref(plan))


def mnb_counters_get():
    c = mnb_counters()
    lib().mnb_counters_get(ctypes.byref(c))
    return c.as_dict()


def mnb_counters_reset():
    lib().mnb_counters_reset()


def mnb_get_kernel_info(m, K, plan):
    info = mnb_kernel_info()
    L = lib()
    _check(L.mnb_get_kernel_info(m, K, ctypes.byref(plan), ctypes.byref(info)), L)
    return info.as_dict()


def mnb_status_string(status):
    return lib().mnb_status_string(status).decode()


def mnb_last_hip_error():
    return lib().mnb_last_hip_error()


def mnb_abi_version():
    return lib().mnb_abi_version()
