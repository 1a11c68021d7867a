"""gdn2 -- Gated Delta Rule-2 kernels for NVIDIA B200 (sm_100a).

Thin Python binding of the C ABI in ``include/gdn2.h``: argument marshalling
only.  Every step of the computation runs in the CUDA library
``_build/libgdn2.so``; PyTorch provides device memory and streams.  There is
no CPU fallback: if the library is missing or no GPU is present the calls
raise.

Entry points (same names as the C ABI):

* :func:`chunk_fwd` -- chunkwise parallel forward over whole sequences
  (``gdn2_chunk_fwd``);
* :func:`chunk_bwd` -- gradients through the chunkwise forward
  (``gdn2_chunk_bwd``);
* :func:`decode_step` -- one recurrent step for a batch of single tokens
  (``gdn2_decode_step``);
* :func:`recurrent_fwd` -- the token loop over whole sequences in either erase orientation
  (``gdn2_recurrent_fwd``);
* :func:`block_prologue`, :func:`block_epilogue` -- the work around the mixer
  in its block (``gdn2_block_prologue``, ``gdn2_block_epilogue``);
* :func:`block_prologue_bwd`, :func:`block_epilogue_bwd` -- gradients through
  them (``gdn2_block_prologue_bwd``, ``gdn2_block_epilogue_bwd``);
* :func:`layer_norm_fwd`, :func:`layer_norm_bwd` -- the norm in front of the
  block's projections (``gdn2_layer_norm_fwd``, ``gdn2_layer_norm_bwd``);
* :func:`act_pack`, :func:`act_unpack`, :class:`Act8` -- activations held in 8
  bits between the forward and the backward pass (``gdn2_act_pack``,
  ``gdn2_act_unpack``), which the backward calls read directly.
"""
import ctypes
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libgdn2.so")

GDN2_OK, GDN2_ERR_INVALID_ARG, GDN2_ERR_UNSUPPORTED, GDN2_ERR_CUDA, GDN2_ERR_TIMEOUT = range(5)
GDN2_F32, GDN2_BF16 = 0, 1
GDN2_ERASE_R1, GDN2_ERASE_R2 = 0, 1
_DTYPES = {torch.float32: GDN2_F32, torch.bfloat16: GDN2_BF16}

_lib = None


class Gdn2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib().gdn2_status_string(status).decode()}")


def lib():
    """The loaded ctypes library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"gdn2 CUDA library not built ({LIB_PATH} missing); "
                               "run `python -m gated_delta_rule_131_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, ci = ctypes.c_void_p, ctypes.c_int
        L.gdn2_chunk_fwd.argtypes = [vp] * 9 + [ci] * 6 + [vp, ci, vp]
        L.gdn2_chunk_fwd.restype = ci
        L.gdn2_chunk_fwd_noalloc.argtypes = [vp] * 9 + [ci] * 6 + [vp, ci, vp]
        L.gdn2_chunk_fwd_noalloc.restype = ci
        L.gdn2_block_prologue.argtypes = [vp] * 15 + [ci] * 6 + [vp, ci, vp]
        L.gdn2_block_prologue.restype = ci
        L.gdn2_block_epilogue.argtypes = [vp] * 4 + [ctypes.c_longlong, ci, ci, ci, vp]
        L.gdn2_block_epilogue.restype = ci
        L.gdn2_decode_step.argtypes = [vp] * 8 + [ci] * 5 + [vp]
        L.gdn2_decode_step.restype = ci
        L.gdn2_status_string.argtypes = [ci]
        L.gdn2_status_string.restype = ctypes.c_char_p
        L.gdn2_device_status.argtypes = [ci]
        L.gdn2_device_status.restype = ci
        L.gdn2_selftest_bounded_wait.argtypes = [ci, vp]
        L.gdn2_selftest_bounded_wait.restype = ci
        L.gdn2_launch_count.argtypes = []
        L.gdn2_chunk_fwd_workspace_bytes.argtypes = [ci] * 7 + [ci]
        L.gdn2_chunk_fwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn2_launch_count.restype = ctypes.c_uint64
        L.gdn2_recurrent_fwd.argtypes = [vp] * 9 + [ci] * 5 + [vp, ci, ci, vp]
        L.gdn2_recurrent_fwd.restype = ci
        L.gdn2_chunk_bwd.argtypes = [vp] * 16 + [ci] * 5 + [vp, ci, vp]
        L.gdn2_chunk_bwd.restype = ci
        L.gdn2_chunk_bwd_workspace_bytes.argtypes = [ci] * 6
        L.gdn2_chunk_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn2_chunk_fwd_plan.argtypes = [ci] * 9 + [ctypes.POINTER(ChunkPlan)]
        L.gdn2_chunk_fwd_plan.restype = ci
        cll = ctypes.c_longlong
        L.gdn2_act_pack.argtypes = [vp] * 5 + [ci, ci, vp]
        L.gdn2_act_pack.restype = ci
        L.gdn2_act_unpack.argtypes = [vp] * 5 + [ci, ci, vp]
        L.gdn2_act_unpack.restype = ci
        L.gdn2_layer_norm_fwd.argtypes = [vp] * 4 + [ctypes.c_float] + [vp] * 6 + [cll, ci, ci, vp]
        L.gdn2_layer_norm_fwd.restype = ci
        L.gdn2_layer_norm_bwd.argtypes = [vp] * 10 + [cll, ci, ci, vp]
        L.gdn2_layer_norm_bwd.restype = ci
        L.gdn2_layer_norm_bwd_workspace_bytes.argtypes = [cll, ci, ci]
        L.gdn2_layer_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn2_block_epilogue_bwd.argtypes = [vp] * 9 + [cll, ci, ci, ci, vp]
        L.gdn2_block_epilogue_bwd.restype = ci
        L.gdn2_block_epilogue_bwd_workspace_bytes.argtypes = [cll, ci, ci, ci]
        L.gdn2_block_epilogue_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn2_block_prologue_bwd.argtypes = [vp] * 25 + [ci] * 6 + [vp, ci, vp]
        L.gdn2_block_prologue_bwd.restype = ci
        L.gdn2_block_prologue_bwd_workspace_bytes.argtypes = [ci] * 8
        L.gdn2_block_prologue_bwd_workspace_bytes.restype = ctypes.c_size_t
        _lib = L
    return _lib


class ChunkPlan(ctypes.Structure):
    """``gdn2_chunk_plan`` of include/gdn2.h."""
    _fields_ = [("records", ctypes.c_longlong), ("wy_ctas", ctypes.c_longlong), ("state_ctas", ctypes.c_longlong),
                ("segments", ctypes.c_int), ("segment_chunks", ctypes.c_int), ("handover_sms", ctypes.c_int),
                ("handover_at", ctypes.c_longlong), ("order", ctypes.c_int), ("launches", ctypes.c_int),
                ("workspace_bytes", ctypes.c_size_t)]


def chunk_fwd_plan(B, T, H, dk, dv, packed=False, sms=0, dtype=torch.bfloat16, chunk=64) -> dict:
    """What a tensor-core ``chunk_fwd`` call of this shape decides before it launches, for a device
    of ``sms`` SMs (0: the current one): records, grids, segments, the SM hand-over, the walking
    order, launches and workspace bytes.  Host only; raises ``Gdn2Error`` when the shape does not
    take the tensor-core path."""
    plan = ChunkPlan()
    st = lib().gdn2_chunk_fwd_plan(B, T, H, dk, dv, chunk, 1 if packed else 0, _DTYPES[dtype], sms, ctypes.byref(plan))
    if st != GDN2_OK:
        raise Gdn2Error(st, "chunk_fwd_plan")
    return {name: int(getattr(plan, name)) for name, _ in ChunkPlan._fields_}


def chunk_fwd_workspace_bytes(B, T, H, dk, dv, packed=False, dtype=torch.bfloat16, chunk=64) -> int:
    """Device bytes ``chunk_fwd`` takes from the library's pool for this shape (0: none)."""
    return int(lib().gdn2_chunk_fwd_workspace_bytes(B, T, H, dk, dv, chunk, 1 if packed else 0, _DTYPES[dtype]))


def launch_count() -> int:
    """Kernel launches issued by the library so far in this process."""
    return int(lib().gdn2_launch_count())


def device_status(reset=False) -> int:
    """Sticky device-side status (GDN2_OK or GDN2_ERR_TIMEOUT); synchronises with the device."""
    return int(lib().gdn2_device_status(1 if reset else 0))


def selftest_bounded_wait(limit_us=20000, stream=None):
    """Run the bounded-wait self-test (a wait that nothing completes gives up after limit_us)."""
    st = lib().gdn2_selftest_bounded_wait(int(limit_us), _stream(stream))
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_selftest_bounded_wait")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None):
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check_tensors(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("gdn2: all tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("gdn2: all tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("gdn2: tensors on different devices")


def _chunk(entry, q, k, v, alpha, b, w, S0, cu_seqlens, chunk, o, S_T, output_final_state, stream):
    if cu_seqlens is None:
        B, T, H, dk = q.shape
    else:
        if cu_seqlens.dtype != torch.int32:
            raise ValueError("gdn2: cu_seqlens must be int32")
        B = cu_seqlens.numel() - 1
        T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DTYPES or any(x.dtype != q.dtype for x in (k, v, alpha, b, w)):
        raise ValueError("gdn2: q, k, v, alpha, b, w must share dtype float32 or bfloat16")
    if o is None:
        o = torch.empty(q.shape[:-1] + (dv,), dtype=q.dtype, device=q.device)
    if S_T is None and output_final_state:
        S_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if S0 is not None and S0.dtype != torch.float32:
        raise ValueError("gdn2: S0 must be float32")
    _check_tensors(q, k, v, alpha, b, w, S0, o, S_T, cu_seqlens)
    fn = getattr(lib(), entry)
    with torch.cuda.device(q.device):  # the library's pool and fixed workspace follow the current device
        st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(o), _ptr(S_T),
                B, T, H, dk, dv, chunk, _ptr(cu_seqlens), _DTYPES[q.dtype], _stream(stream, q.device))
    if st != GDN2_OK:
        raise Gdn2Error(st, entry)
    return o, S_T


def chunk_fwd(q, k, v, alpha, b, w, S0=None, cu_seqlens=None, chunk=64, o=None, S_T=None,
              output_final_state=True, stream=None):
    """Chunkwise forward.  Returns ``(o, S_T)`` (``S_T`` None if not requested).

    Dense: q, k, alpha, b ``[B, T, H, d_k]``; v, w ``[B, T, H, d_v]``.
    Packed (``cu_seqlens`` int32 ``[N+1]`` on the device): ``[T_total, H, d]``.
    ``S0`` / ``S_T``: ``[N, H, d_k, d_v]`` float32.
    """
    return _chunk("gdn2_chunk_fwd", q, k, v, alpha, b, w, S0, cu_seqlens, chunk, o, S_T,
                  output_final_state, stream)


def chunk_fwd_noalloc(q, k, v, alpha, b, w, S0=None, cu_seqlens=None, chunk=64, o=None, S_T=None,
                      output_final_state=True, stream=None):
    """``chunk_fwd`` through the library's fixed workspace: the library allocates nothing.

    For callers that cannot let the library allocate device memory (all memory reserved up front,
    or owned by the caller's own memory manager).  The first call on a device looks the fixed
    array's address up; make it before any stream capture.  Shapes whose workspace exceeds
    ``NOALLOC_WORKSPACE_BYTES`` raise ``Gdn2Error`` (``GDN2_ERR_UNSUPPORTED``).  Calls that overlap
    in time on one device race on the shared workspace; calls on one stream are ordered.
    """
    return _chunk("gdn2_chunk_fwd_noalloc", q, k, v, alpha, b, w, S0, cu_seqlens, chunk, o, S_T,
                  output_final_state, stream)


NOALLOC_WORKSPACE_BYTES = 64 << 20  # GDN2_NOALLOC_WORKSPACE_BYTES in include/gdn2.h


def recurrent_fwd(q, k, v, alpha, b, w, S0=None, cu_seqlens=None, erase=GDN2_ERASE_R1, o=None, S_T=None,
                  output_final_state=True, stream=None):
    """Token-by-token forward in either erase orientation (``GDN2_ERASE_R1`` or ``GDN2_ERASE_R2``).

    Same layouts and returns as :func:`chunk_fwd`; see ``gdn2_recurrent_fwd`` in ``include/gdn2.h``.
    """
    if cu_seqlens is None:
        B, T, H, dk = q.shape
    else:
        if cu_seqlens.dtype != torch.int32:
            raise ValueError("gdn2: cu_seqlens must be int32")
        B = cu_seqlens.numel() - 1
        T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DTYPES or any(x.dtype != q.dtype for x in (k, v, alpha, b, w)):
        raise ValueError("gdn2: q, k, v, alpha, b, w must share dtype float32 or bfloat16")
    if o is None:
        o = torch.empty(q.shape[:-1] + (dv,), dtype=q.dtype, device=q.device)
    if S_T is None and output_final_state:
        S_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if S0 is not None and S0.dtype != torch.float32:
        raise ValueError("gdn2: S0 must be float32")
    _check_tensors(q, k, v, alpha, b, w, S0, o, S_T, cu_seqlens)
    with torch.cuda.device(q.device):
        st = lib().gdn2_recurrent_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(o),
                                      _ptr(S_T), B, T, H, dk, dv, _ptr(cu_seqlens), int(erase), _DTYPES[q.dtype],
                                      _stream(stream, q.device))
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_recurrent_fwd")
    return o, S_T


def chunk_bwd(q, k, v, alpha, b, w, dO, S0=None, dS_T=None, cu_seqlens=None, want_dS0=True, stream=None):
    """Gradients of a loss through ``chunk_fwd`` given ``dO = dL/do`` and ``dS_T = dL/dS_T`` (or None).

    Returns ``(dq, dk, dv, dalpha, db, dw, dS0)`` in the layouts and dtype of the inputs (``dS0``
    float32 ``[N, H, d_k, d_v]``, None unless ``want_dS0``).  See ``gdn2_chunk_bwd`` in ``include/gdn2.h``.
    """
    if cu_seqlens is None:
        B, T, H, dk = q.shape
    else:
        if cu_seqlens.dtype != torch.int32:
            raise ValueError("gdn2: cu_seqlens must be int32")
        B = cu_seqlens.numel() - 1
        T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DTYPES or any(x.dtype != q.dtype for x in (k, v, alpha, b, w, dO)):
        raise ValueError("gdn2: q, k, v, alpha, b, w, dO must share dtype float32 or bfloat16")
    if any(x is not None and x.dtype != torch.float32 for x in (S0, dS_T)):
        raise ValueError("gdn2: S0 and dS_T must be float32")
    grads = [torch.empty_like(x) for x in (q, k, v, alpha, b, w)]
    dS0 = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device) if want_dS0 else None
    _check_tensors(q, k, v, alpha, b, w, dO, S0, dS_T, *grads, dS0, cu_seqlens)
    with torch.cuda.device(q.device):
        st = lib().gdn2_chunk_bwd(*[_ptr(x) for x in (q, k, v, alpha, b, w, S0, dO, dS_T)],
                                  *[_ptr(x) for x in grads], _ptr(dS0), B, T, H, dk, dv, _ptr(cu_seqlens),
                                  _DTYPES[q.dtype], _stream(stream, q.device))
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_chunk_bwd")
    dq, dk_, dv_, dalpha, db, dw = grads
    return dq, dk_, dv_, dalpha, db, dw, dS0


def chunk_bwd_workspace_bytes(B, T, H, d_k, d_v, packed=False):
    """Device bytes ``chunk_bwd`` takes from the library's pool for this shape."""
    return int(lib().gdn2_chunk_bwd_workspace_bytes(B, T, H, d_k, d_v, int(bool(packed))))


def block_prologue(xq, xk, xv, xa, xb, xw, conv_q, conv_k, conv_v, cu_seqlens=None, stream=None):
    """The mixer's inputs from the projections' outputs: returns ``(q, k, v, alpha, b, w)``.

    Token tensors ``[B, T, H, d]`` (dense) or ``[T_total, H, d]`` with ``cu_seqlens``; convolution
    weights ``[H*d, K]`` float32 with K in 1..4.  See ``gdn2_block_prologue`` in ``include/gdn2.h``.
    """
    if cu_seqlens is None:
        B, T, H, dk = xq.shape
    else:
        if cu_seqlens.dtype != torch.int32:
            raise ValueError("gdn2: cu_seqlens must be int32")
        B = cu_seqlens.numel() - 1
        T, H, dk = xq.shape
    dv = xv.shape[-1]
    if xq.dtype not in _DTYPES or any(x.dtype != xq.dtype for x in (xk, xv, xa, xb, xw)):
        raise ValueError("gdn2: the pre-activations must share dtype float32 or bfloat16")
    if any(W.dtype != torch.float32 for W in (conv_q, conv_k, conv_v)):
        raise ValueError("gdn2: convolution weights must be float32")
    outs = [torch.empty_like(x) for x in (xq, xk, xv, xa, xb, xw)]
    _check_tensors(xq, xk, xv, xa, xb, xw, conv_q, conv_k, conv_v, *outs, cu_seqlens)
    with torch.cuda.device(xq.device):
        st = lib().gdn2_block_prologue(*[_ptr(x) for x in (xq, xk, xv, xa, xb, xw, conv_q, conv_k, conv_v)],
                                       *[_ptr(x) for x in outs], B, T, H, dk, dv, conv_q.shape[1],
                                       _ptr(cu_seqlens), _DTYPES[xq.dtype], _stream(stream, xq.device))
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_block_prologue")
    return tuple(outs)


def block_epilogue(o, gate, norm_weight, y=None, stream=None):
    """``y = RMSNorm(o) * norm_weight * SiLU(gate)`` per (token, head) over d_v; ``y`` may be ``o``."""
    H, dv = o.shape[-2], o.shape[-1]
    tokens = o.numel() // (H * dv)
    if o.dtype not in _DTYPES or gate.dtype != o.dtype:
        raise ValueError("gdn2: o and gate must share dtype float32 or bfloat16")
    if norm_weight.dtype != torch.float32:
        raise ValueError("gdn2: norm_weight must be float32")
    if y is None:
        y = torch.empty_like(o)
    _check_tensors(o, gate, norm_weight, y)
    with torch.cuda.device(o.device):
        st = lib().gdn2_block_epilogue(_ptr(o), _ptr(gate), _ptr(norm_weight), _ptr(y), tokens, H, dv,
                                       _DTYPES[o.dtype], _stream(stream, o.device))
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_block_epilogue")
    return y


def decode_step(q, k, v, alpha, b, w, S, o=None, stream=None):
    """One decode step: updates ``S`` ``[B, H, d_k, d_v]`` in place, returns ``o`` ``[B, H, d_v]``."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DTYPES or any(x.dtype != q.dtype for x in (k, v, alpha, b, w)):
        raise ValueError("gdn2: q, k, v, alpha, b, w must share dtype float32 or bfloat16")
    if S.dtype != torch.float32:
        raise ValueError("gdn2: S must be float32")
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    _check_tensors(q, k, v, alpha, b, w, S, o)
    with torch.cuda.device(q.device):
        st = lib().gdn2_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b), _ptr(w), _ptr(S),
                                    _ptr(o), B, H, dk, dv, _DTYPES[q.dtype], _stream(stream, q.device))
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_decode_step")
    return o


# ------------------------------------------------------------------------------------------------
# training operators of the block

ACT_GROUP = 32          # channels that share a scale in an Act8
ACT_MAX_TENSORS = 8     # GDN2_ACT_MAX_TENSORS in include/gdn2.h
NORM_MAX_WIDTH = 8192   # GDN2_NORM_MAX_WIDTH in include/gdn2.h
_INT_MAX = 2 ** 31 - 1  # the C ABI's sizes are ints; ctypes would cut larger ones to their low 32 bits


class Act8(NamedTuple):
    """A tensor held in 8 bits: ``codes`` int8 in its shape, ``scales`` uint8 ``[..., ceil(D / 32)]``
    for its last dimension ``D`` (the format is described in ``include/gdn2.h``)."""
    codes: torch.Tensor
    scales: torch.Tensor


class LayerNormOut(NamedTuple):
    """What :func:`layer_norm_fwd` returns; ``checkpoint`` is ``h`` as an :class:`Act8`, or None."""
    y: torch.Tensor
    h: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    checkpoint: Optional[Act8]


def _handle(tensors):
    """The handle of the current stream, or None where the tensors' device is not the current one.
    (Everything on this path is paid by every call, short ones too, so it is kept plain.)"""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError("gdn2: all tensors must be CUDA tensors")
                if dev is not None:
                    raise ValueError("gdn2: tensors on different devices")
                dev = d
            if not t.is_contiguous():
                raise ValueError("gdn2: all tensors must be contiguous")
    if dev != torch.cuda.current_device():
        return None
    return torch._C._cuda_getCurrentRawStream(dev)


def _elsewhere(stream, tensors, call):
    """``call()`` with the tensors' device and ``stream`` (None: that device's current one) made current:
    outputs are allocated for that stream, and inputs are kept until its work is done."""
    tensors = [t for t in tensors if t is not None]
    _check_tensors(*tensors)
    dev = tensors[0].device
    if stream is not None and stream.device != dev:
        raise ValueError("gdn2: the stream is on another device than the tensors")
    with torch.cuda.device(dev):
        if stream is None or stream == torch.cuda.current_stream(dev):
            return call()
        with torch.cuda.stream(stream):
            out = call()
        for t in tensors:
            t.record_stream(stream)
        return out


def _expect(what, name, t, dtype, shape):
    if t is None:
        raise ValueError(f"gdn2: {what}: {name} is missing")
    if t.dtype is dtype and t.shape == shape:
        return
    raise ValueError(f"gdn2: {what}: {name} must be {dtype} of shape {tuple(shape)}, not {t.dtype} of {tuple(t.shape)}")


def _addr(t):
    return None if t is None else t.data_ptr()


def _act8_shape(shape):
    return (*shape[:-1], -(-shape[-1] // ACT_GROUP))


def _check_act8(what, name, a, shape):
    _expect(what, name + ".codes", a.codes, torch.int8, shape)
    _expect(what, name + ".scales", a.scales, torch.uint8, _act8_shape(shape))


def _new_act8(x):
    return Act8(torch.empty_like(x, dtype=torch.int8), x.new_empty(_act8_shape(x.shape), dtype=torch.uint8))


def _saved(what, name, x, like):
    """A saved activation as (values or codes, scales or None), checked against its gradient."""
    if isinstance(x, Act8):
        _check_act8(what, name, x, like.shape)
        return x.codes, x.scales
    _expect(what, name, x, like.dtype, like.shape)
    return x, None


_HOST_ARRAYS = [(ctypes.c_void_p * n, ctypes.c_longlong * n, ctypes.c_int * n) for n in range(ACT_MAX_TENSORS + 1)]


def _act_call(entry, first, second, third, dtype, stream):
    """``first`` holds tensors of the shapes of the values."""
    n = len(first)
    if n > ACT_MAX_TENSORS:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, entry)
    pointers, longs, ints = _HOST_ARRAYS[n]
    width = [t.shape[-1] for t in first]
    st = getattr(lib(), entry)(pointers(*[t.data_ptr() for t in first]), pointers(*[t.data_ptr() for t in second]),
                               pointers(*[t.data_ptr() for t in third]),
                               longs(*[t.numel() // w for t, w in zip(first, width)]), ints(*width), n,
                               _DTYPES[dtype], stream)
    if st != GDN2_OK:
        raise Gdn2Error(st, entry)


def act_pack(xs, stream=None):
    """Hold a tensor, or a list of up to ``ACT_MAX_TENSORS`` of one dtype, in 8 bits: returns an
    :class:`Act8` or a list of them.  See ``gdn2_act_pack`` in ``include/gdn2.h``."""
    one = isinstance(xs, torch.Tensor)
    xs = [xs] if one else list(xs)
    if not xs:
        return []
    dtype = xs[0].dtype
    for x in xs:
        if x.dtype is not dtype or dtype not in _DTYPES:
            raise ValueError("gdn2: act_pack: the tensors must share dtype float32 or bfloat16")
        if x.dim() < 1 or not 1 <= x.shape[-1] <= _INT_MAX:
            raise ValueError("gdn2: act_pack: a tensor needs a last dimension of 1 to 2^31 - 1")
    s = _handle(xs) if stream is None else None
    if s is None:
        return _elsewhere(stream, xs, lambda: act_pack(xs[0] if one else xs))
    out = [_new_act8(x) for x in xs]
    _act_call("gdn2_act_pack", xs, [a.codes for a in out], [a.scales for a in out], dtype, s)
    return out[0] if one else out


def act_unpack(acts, dtype=torch.bfloat16, stream=None):
    """The values that an :class:`Act8`, or a list of them, holds (exact in either dtype)."""
    one = isinstance(acts, Act8)
    acts = [acts] if one else list(acts)
    if not acts:
        return []
    if dtype not in _DTYPES:
        raise ValueError("gdn2: act_unpack: dtype must be float32 or bfloat16")
    for a in acts:
        if a.codes.dim() < 1 or not 1 <= a.codes.shape[-1] <= _INT_MAX:
            raise ValueError("gdn2: act_unpack: a tensor needs a last dimension of 1 to 2^31 - 1")
        _check_act8("act_unpack", "act", a, a.codes.shape)
    codes, scales = [a.codes for a in acts], [a.scales for a in acts]
    s = _handle(codes + scales) if stream is None else None
    if s is None:
        return _elsewhere(stream, codes + scales, lambda: act_unpack(acts[0] if one else acts, dtype))
    out = [torch.empty_like(c, dtype=dtype) for c in codes]
    _act_call("gdn2_act_unpack", codes, scales, out, dtype, s)
    return out[0] if one else out


def layer_norm_fwd(x, weight, bias=None, residual=None, eps=1e-5, checkpoint=False, stats=True, stream=None):
    """Layer norm over the last dimension, of ``h = x + residual``: returns a :class:`LayerNormOut`.

    ``h`` is ``x`` itself without a residual; ``mean`` and ``rstd`` (float32, one per row) are None
    with ``stats=False``; ``checkpoint=True`` also returns ``h`` held in 8 bits.  See
    ``gdn2_layer_norm_fwd`` in ``include/gdn2.h``.
    """
    what, shape, dtype = "layer_norm_fwd", x.shape, x.dtype
    if dtype not in _DTYPES:
        raise ValueError("gdn2: layer_norm_fwd: x must be float32 or bfloat16")
    if not shape or shape[-1] < 1:
        raise ValueError("gdn2: layer_norm_fwd: x needs a last dimension of at least 1")
    D = shape[-1]
    if D > NORM_MAX_WIDTH:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, "gdn2_layer_norm_fwd")
    if residual is not None:
        _expect(what, "residual", residual, dtype, shape)
    _expect(what, "weight", weight, torch.float32, (D,))
    if bias is not None:
        _expect(what, "bias", bias, torch.float32, (D,))
    tensors = (x, weight, bias, residual)
    s = _handle(tensors) if stream is None else None
    if s is None:
        return _elsewhere(stream, tensors, lambda: layer_norm_fwd(x, weight, bias, residual, eps, checkpoint, stats))
    y = torch.empty_like(x)
    h = mean = rstd = ck = codes = scales = None
    if residual is not None:
        h = torch.empty_like(x)
    if stats:
        mean = x.new_empty(shape[:-1], dtype=torch.float32)
        rstd = torch.empty_like(mean)
    if checkpoint:
        codes, scales = ck = _new_act8(x)
    st = lib().gdn2_layer_norm_fwd(x.data_ptr(), _addr(residual), weight.data_ptr(), _addr(bias), eps, y.data_ptr(),
                                   _addr(h), _addr(mean), _addr(rstd), _addr(codes), _addr(scales), x.numel() // D, D,
                                   _DTYPES[dtype], s)
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_layer_norm_fwd")
    return LayerNormOut(y, x if h is None else h, mean, rstd, ck)


def layer_norm_bwd(dy, h, mean, rstd, weight, dh=None, want_dbias=True, stream=None):
    """Gradients through :func:`layer_norm_fwd`: ``(dx, dweight, dbias)``, ``dx`` being the gradient of
    ``x`` and of ``residual``, with ``dh`` (the gradient that reaches ``h`` past the norm) added.

    ``h`` is the forward's ``h`` or its :class:`Act8` checkpoint.  ``dbias`` is None unless
    ``want_dbias``.  See ``gdn2_layer_norm_bwd`` in ``include/gdn2.h``.
    """
    what, shape, dtype = "layer_norm_bwd", dy.shape, dy.dtype
    if dtype not in _DTYPES:
        raise ValueError("gdn2: layer_norm_bwd: dy must be float32 or bfloat16")
    if not shape or shape[-1] < 1:
        raise ValueError("gdn2: layer_norm_bwd: dy needs a last dimension of at least 1")
    D = shape[-1]
    if D > NORM_MAX_WIDTH:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, "gdn2_layer_norm_bwd")
    if dh is not None:
        _expect(what, "dh", dh, dtype, shape)
    _expect(what, "mean", mean, torch.float32, shape[:-1])
    _expect(what, "rstd", rstd, torch.float32, shape[:-1])
    _expect(what, "weight", weight, torch.float32, (D,))
    values, scales = _saved(what, "h", h, dy)
    tensors = (dy, values, scales, mean, rstd, weight, dh)
    s = _handle(tensors) if stream is None else None
    if s is None:
        return _elsewhere(stream, tensors, lambda: layer_norm_bwd(dy, h, mean, rstd, weight, dh, want_dbias))
    dx, dweight = torch.empty_like(dy), torch.empty_like(weight)
    dbias = torch.empty_like(weight) if want_dbias else None
    st = lib().gdn2_layer_norm_bwd(dy.data_ptr(), values.data_ptr(), _addr(scales), mean.data_ptr(), rstd.data_ptr(),
                                   weight.data_ptr(), _addr(dh), dx.data_ptr(), dweight.data_ptr(), _addr(dbias),
                                   dy.numel() // D, D, _DTYPES[dtype], s)
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_layer_norm_bwd")
    return dx, dweight, dbias


def layer_norm_bwd_workspace_bytes(tokens, width, dtype=torch.bfloat16) -> int:
    """Device bytes ``layer_norm_bwd`` takes from the library's pool for this shape (0: none, or a shape
    that it does not take)."""
    if abs(width) > _INT_MAX:
        return 0
    return int(lib().gdn2_layer_norm_bwd_workspace_bytes(tokens, width, _DTYPES[dtype]))


def block_epilogue_bwd(o, gate, norm_weight, dy, stream=None):
    """Gradients through :func:`block_epilogue`: ``(do, dgate, dnorm_weight)``.

    ``o`` and ``gate`` are the forward's inputs, or both :class:`Act8` checkpoints of them.  See
    ``gdn2_block_epilogue_bwd`` in ``include/gdn2.h``.
    """
    what, shape, dtype = "block_epilogue_bwd", dy.shape, dy.dtype
    if dtype not in _DTYPES:
        raise ValueError("gdn2: block_epilogue_bwd: dy must be float32 or bfloat16")
    if len(shape) < 2 or shape[-2] < 1 or shape[-1] < 1:
        raise ValueError("gdn2: block_epilogue_bwd: dy must be [..., H, d_v]")
    if isinstance(o, Act8) != isinstance(gate, Act8):
        raise ValueError("gdn2: block_epilogue_bwd: o and gate are both tensors or both Act8")
    H, dv = shape[-2], shape[-1]
    if H > _INT_MAX or dv > _INT_MAX:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, "gdn2_block_epilogue_bwd")
    _expect(what, "norm_weight", norm_weight, torch.float32, (dv,))
    oc, osc = _saved(what, "o", o, dy)
    gc, gsc = _saved(what, "gate", gate, dy)
    tensors = (oc, osc, gc, gsc, norm_weight, dy)
    s = _handle(tensors) if stream is None else None
    if s is None:
        return _elsewhere(stream, tensors, lambda: block_epilogue_bwd(o, gate, norm_weight, dy))
    do, dgate, dnorm_weight = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(norm_weight)
    st = lib().gdn2_block_epilogue_bwd(oc.data_ptr(), gc.data_ptr(), _addr(osc), _addr(gsc), norm_weight.data_ptr(),
                                       dy.data_ptr(), do.data_ptr(), dgate.data_ptr(), dnorm_weight.data_ptr(),
                                       dy.numel() // (H * dv), H, dv, _DTYPES[dtype], s)
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_block_epilogue_bwd")
    return do, dgate, dnorm_weight


def block_epilogue_bwd_workspace_bytes(tokens, H, d_v, dtype=torch.bfloat16) -> int:
    """Device bytes ``block_epilogue_bwd`` takes from the library's pool for this shape (0: none, or a
    shape that it does not take)."""
    if max(abs(H), abs(d_v)) > _INT_MAX:
        return 0
    return int(lib().gdn2_block_epilogue_bwd_workspace_bytes(tokens, H, d_v, _DTYPES[dtype]))


_PRE = ("xq", "xk", "xv", "xa", "xb", "xw")


def block_prologue_bwd(xq, xk, xv, xa, xb, xw, conv_q, conv_k, conv_v, dq, dk, dv, dalpha, db, dw, cu_seqlens=None,
                       stream=None):
    """Gradients through :func:`block_prologue` from those that :func:`chunk_bwd` returns:
    ``(dxq, dxk, dxv, dxa, dxb, dxw, dconv_q, dconv_k, dconv_v)``.

    The six inputs are the forward's, or all :class:`Act8` checkpoints of them.  In a packed batch,
    rows behind the last sequence keep whatever memory their gradients were given.  See
    ``gdn2_block_prologue_bwd`` in ``include/gdn2.h``.
    """
    what, shape, dtype = "block_prologue_bwd", dq.shape, dq.dtype
    xs, grads, convs = (xq, xk, xv, xa, xb, xw), (dq, dk, dv, dalpha, db, dw), (conv_q, conv_k, conv_v)
    if dtype not in _DTYPES:
        raise ValueError("gdn2: block_prologue_bwd: the gradients must be float32 or bfloat16")
    packed8 = isinstance(xq, Act8)
    for x in xs:
        if isinstance(x, Act8) != packed8:
            raise ValueError("gdn2: block_prologue_bwd: the saved inputs are all tensors or all Act8")
    if dv is None or conv_q is None:
        raise ValueError("gdn2: block_prologue_bwd: dv and conv_q are needed")
    if len(shape) != (4 if cu_seqlens is None else 3) or not dv.shape or conv_q.dim() != 2:
        raise ValueError("gdn2: block_prologue_bwd: gradients are [B, T, H, d], or [T, H, d] with cu_seqlens; "
                         "convolution weights [H * d, K]")
    if cu_seqlens is None:
        B, T, H, d_k = shape
    else:
        if cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("gdn2: block_prologue_bwd: cu_seqlens must be int32 [B + 1]")
        B = cu_seqlens.numel() - 1
        T, H, d_k = shape
    d_v, K = dv.shape[-1], conv_q.shape[1]
    if max(B, T, H, d_k, d_v, K) > _INT_MAX:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, "gdn2_block_prologue_bwd")
    vshape = torch.Size((*shape[:-1], d_v))
    shapes = (shape, shape, vshape, shape, shape, vshape)
    for i in range(6):
        if grads[i] is None or grads[i].dtype is not dtype or grads[i].shape != shapes[i]:
            _expect(what, ("dq", "dk", "dv", "dalpha", "db", "dw")[i], grads[i], dtype, shapes[i])
        if packed8:
            _check_act8(what, _PRE[i], xs[i], shapes[i])
        elif xs[i] is None or xs[i].dtype is not dtype or xs[i].shape != shapes[i]:
            _expect(what, _PRE[i], xs[i], dtype, shapes[i])
    for i, d in enumerate((d_k, d_k, d_v)):
        _expect(what, ("conv_q", "conv_k", "conv_v")[i], convs[i], torch.float32, (H * d, K))
    saved, scale_list = ([x.codes for x in xs], [x.scales for x in xs]) if packed8 else (xs, ())
    tensors = (*grads, *saved, *scale_list, *convs, cu_seqlens)
    s = _handle(tensors) if stream is None else None
    if s is None:
        return _elsewhere(stream, tensors, lambda: block_prologue_bwd(*xs, *convs, *grads, cu_seqlens=cu_seqlens))
    dxs = [torch.empty_like(t) for t in grads]
    dconv = [torch.empty_like(t) for t in convs]
    scales = _HOST_ARRAYS[6][0](*[t.data_ptr() for t in scale_list]) if packed8 else None
    st = lib().gdn2_block_prologue_bwd(*[t.data_ptr() for t in saved], scales, *[t.data_ptr() for t in convs],
                                       *[t.data_ptr() for t in grads], *[t.data_ptr() for t in dxs],
                                       *[t.data_ptr() for t in dconv], B, T, H, d_k, d_v, K, _addr(cu_seqlens),
                                       _DTYPES[dtype], s)
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_block_prologue_bwd")
    return (*dxs, *dconv)


def block_prologue_bwd_workspace_bytes(B, T, H, d_k, d_v, conv_len, packed=False, dtype=torch.bfloat16) -> int:
    """Device bytes ``block_prologue_bwd`` takes from the library's pool for this shape (0: a shape that it
    does not take)."""
    if max(abs(n) for n in (B, T, H, d_k, d_v, conv_len)) > _INT_MAX:
        return 0
    return int(lib().gdn2_block_prologue_bwd_workspace_bytes(B, T, H, d_k, d_v, conv_len, int(bool(packed)),
                                                             _DTYPES[dtype]))
