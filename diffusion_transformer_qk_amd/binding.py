"""ctypes binding of ``libqknorm_rope.so`` (argument marshalling only).

Every step runs in the HIP kernels behind the C ABI declared in
``include/qknorm_rope.h`` (fused QK-norm + RoPE), ``include/fuse_scale_shift.h``
(AdaLN modulation), ``include/group_norm_silu.h`` (group norm + SiLU),
``include/dit_attention.h`` (attention, of padded samples and of packed
sequences, and its backward pass),
``include/layer_norm.h`` (layer norm and its backward pass),
``include/rms_norm.h`` (RMS norm with the residual and an 8-bit output, and its
backward pass), ``include/feed_forward.h`` (the gated feed-forward projection
and its backward pass) and ``include/qknorm_rope_backward.h``;
this module turns torch
tensors into device pointers, sizes and enum codes and raises on a non-zero
status.  There is no fallback: if the library is missing, loading fails
loudly.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqknorm_rope.so")

QKR_OK = 0
QKR_ERR_NULL, QKR_ERR_SHAPE, QKR_ERR_ALIGN = -1, -2, -3
QKR_ERR_UNSUPPORTED, QKR_ERR_MODE, QKR_ERR_HIP, QKR_ERR_ARG = -4, -5, -6, -7
QKR_ERR_WORKSPACE = -8
QKR_ERR_SCRATCH = -9
GN_NOALLOC_WORKSPACE_MAX = 1 << 20
QKR_BF16, QKR_FP16, QKR_FP32 = 0, 1, 2
QKR_COS_SHARED, QKR_COS_PER_HEAD = 0, 1
QKR_ROPE_INTERLEAVED, QKR_ROPE_ROTATE_HALF = 0, 1
QKR_TENSORS_FUSED, QKR_TENSORS_PAIR, QKR_TENSORS_ONE = 0, 1, 2

DIT_FF_E4M3 = 8
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}
LAYOUTS = {"shared": QKR_COS_SHARED, "per_head": QKR_COS_PER_HEAD}
DIT_LN_WEIGHT, DIT_LN_ONE_PLUS = 0, 1
STYLES = {"interleaved": QKR_ROPE_INTERLEAVED, "rotate_half": QKR_ROPE_ROTATE_HALF}
TENSORS = {"fused": QKR_TENSORS_FUSED, "pair": QKR_TENSORS_PAIR, "one": QKR_TENSORS_ONE}
EXPORTS = ("qknorm_rope_fused", "qknorm_rope_strerror", "qknorm_rope_version",
           "qknorm_rope_kernel_info", "dit_fuse_scale_shift",
           "dit_group_norm_silu_workspace_size", "dit_group_norm_silu_schedule",
           "dit_group_norm_silu", "dit_group_norm_silu_noalloc",
           "dit_attention_workspace_size", "dit_attention_backward_workspace_size",
           "dit_attention", "dit_attention_backward", "dit_layer_norm",
           "dit_layer_norm_backward_workspace_size", "dit_layer_norm_backward",
           "qknorm_rope_backward_workspace_size", "qknorm_rope_backward", "dit_rms_norm",
           "dit_rms_norm_backward_workspace_size", "dit_rms_norm_backward",
           "dit_gated_feed_forward", "dit_gated_feed_forward_backward_workspace_size",
           "dit_gated_feed_forward_backward",
           "dit_attention_packed_workspace_size", "dit_attention_packed_backward_workspace_size",
           "dit_attention_packed", "dit_attention_packed_backward")
MOD_DTYPES = {"bf16": QKR_BF16, "fp16": QKR_FP16, "fp32": QKR_FP32}


class QkrError(RuntimeError):
    """A non-zero status from the library."""

    def __init__(self, status: int, message: str):
        super().__init__("qknorm_rope: %s (status %d)" % (message, status))
        self.status = status


class KernelInfo(ctypes.Structure):
    _fields_ = [("num_vgprs", ctypes.c_int32), ("lds_bytes", ctypes.c_int32),
                ("scratch_bytes", ctypes.c_int32), ("block_threads", ctypes.c_int32),
                ("tokens_per_block", ctypes.c_int32), ("heads_in_flight", ctypes.c_int32),
                ("die_runs", ctypes.c_int32), ("dynamic_lds_bytes", ctypes.c_int32),
                ("workgroups_per_cu", ctypes.c_int32)]


class GradTensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("x", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class AttnTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class AttnArgs(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("q_tokens", ctypes.c_int64),
                ("kv_tokens", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("kv_lengths", ctypes.c_void_p)]


class AttnPackedArgs(ctypes.Structure):
    _fields_ = [("sequences", ctypes.c_int64), ("q_tokens", ctypes.c_int64),
                ("kv_tokens", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("fill_rest", ctypes.c_int32), ("q_offsets", ctypes.c_void_p),
                ("kv_offsets", ctypes.c_void_p)]


class FfArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("hidden", ctypes.c_int32), ("inner", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            "libqknorm_rope.so is not built (%s); run __graft_entry__.build() or "
            "python -m diffusion_transformer_qk_amd.build" % path)
    # torch first: it carries its own HIP runtime, and the library's HIP
    # dependency must resolve to that one.  Loaded the other way round, the
    # process holds two runtimes and the library's sees no device.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    lib.qknorm_rope_fused.argtypes = [vp, vp, vp, i64, i32, i32, vp, vp, f32, vp, vp,
                                      i32, i32, i32, i32, vp]
    lib.qknorm_rope_fused.restype = ctypes.c_int
    lib.qknorm_rope_strerror.argtypes = [ctypes.c_int]
    lib.qknorm_rope_strerror.restype = ctypes.c_char_p
    lib.qknorm_rope_version.argtypes = []
    lib.qknorm_rope_version.restype = ctypes.c_int
    lib.qknorm_rope_kernel_info.argtypes = [i32, i32, i64, i32, i32, i32, i32, i32,
                                            ctypes.POINTER(KernelInfo)]
    lib.qknorm_rope_kernel_info.restype = ctypes.c_int
    lib.dit_fuse_scale_shift.argtypes = [vp, vp, i64, i32, i64, vp, vp, i32, f32, i32, vp]
    lib.dit_fuse_scale_shift.restype = ctypes.c_int
    lib.dit_group_norm_silu_workspace_size.argtypes = [i64, i32, i64, i32]
    lib.dit_group_norm_silu_workspace_size.restype = i64
    lib.dit_group_norm_silu_schedule.argtypes = [i64, i32, i64, i32, ctypes.POINTER(i64)]
    lib.dit_group_norm_silu_schedule.restype = i32
    lib.dit_group_norm_silu.argtypes = [vp, vp, i64, i32, i64, i32, vp, vp, i32, f32, i32, vp, i64,
                                        vp]
    lib.dit_group_norm_silu.restype = ctypes.c_int
    lib.dit_group_norm_silu_noalloc.argtypes = [vp, vp, i64, i32, i64, i32, vp, vp, i32, f32,
                                                i32, vp]
    lib.dit_group_norm_silu_noalloc.restype = ctypes.c_int
    args, tensor = ctypes.POINTER(AttnArgs), ctypes.POINTER(AttnTensor)
    for name in ("dit_attention_workspace_size", "dit_attention_backward_workspace_size"):
        getattr(lib, name).argtypes = [args]
        getattr(lib, name).restype = i64
    lib.dit_attention.argtypes = [args, *[tensor] * 4, vp, vp, i64, vp]
    lib.dit_attention.restype = ctypes.c_int
    lib.dit_attention_backward.argtypes = [args, *[tensor] * 5, vp, *[tensor] * 3, vp, i64, vp]
    lib.dit_attention_backward.restype = ctypes.c_int
    packed = ctypes.POINTER(AttnPackedArgs)
    for name in ("dit_attention_packed_workspace_size", "dit_attention_packed_backward_workspace_size"):
        getattr(lib, name).argtypes = [packed]
        getattr(lib, name).restype = i64
    lib.dit_attention_packed.argtypes = [packed, *[tensor] * 4, vp, vp, i64, vp]
    lib.dit_attention_packed.restype = ctypes.c_int
    lib.dit_attention_packed_backward.argtypes = [packed, *[tensor] * 5, vp, *[tensor] * 3, vp, i64, vp]
    lib.dit_attention_packed_backward.restype = ctypes.c_int
    lib.dit_layer_norm.argtypes = [vp, vp, i64, i32, vp, vp, i32, f32, i32, vp]
    lib.dit_layer_norm.restype = ctypes.c_int
    lib.dit_layer_norm_backward_workspace_size.argtypes = [i64, i32, i64]
    lib.dit_layer_norm_backward_workspace_size.restype = i64
    lib.dit_layer_norm_backward.argtypes = [vp, vp, vp, i64, i32, i64, vp, i32, i32, vp, vp, f32,
                                            i32, vp, i64, vp]
    lib.dit_layer_norm_backward.restype = ctypes.c_int
    lib.dit_rms_norm.argtypes = [vp, vp, vp, vp, vp, i64, i32, vp, i32, f32, i32, vp]
    lib.dit_rms_norm.restype = ctypes.c_int
    lib.dit_rms_norm_backward_workspace_size.argtypes = [i64, i32]
    lib.dit_rms_norm_backward_workspace_size.restype = i64
    lib.dit_rms_norm_backward.argtypes = [vp, vp, vp, vp, i64, i32, vp, i32, vp, f32, i32, vp, i64, vp]
    lib.dit_rms_norm_backward.restype = ctypes.c_int
    ff = ctypes.POINTER(FfArgs)
    lib.dit_gated_feed_forward_backward_workspace_size.argtypes = [ff]
    lib.dit_gated_feed_forward_backward_workspace_size.restype = i64
    lib.dit_gated_feed_forward.argtypes = [ff, *[vp] * 10]
    lib.dit_gated_feed_forward.restype = ctypes.c_int
    lib.dit_gated_feed_forward_backward.argtypes = [ff, *[vp] * 10, i64, vp]
    lib.dit_gated_feed_forward_backward.restype = ctypes.c_int
    grad = ctypes.POINTER(GradTensor)
    lib.qknorm_rope_backward_workspace_size.argtypes = [i64, i32]
    lib.qknorm_rope_backward_workspace_size.restype = i64
    lib.qknorm_rope_backward.argtypes = [grad, grad, grad, i64, i32, i32, vp, vp, vp, vp, f32, vp, vp,
                                         i32, i32, i32, i32, vp, i64, vp]
    lib.qknorm_rope_backward.restype = ctypes.c_int
    _lib = lib
    return lib


def strerror(status: int) -> str:
    return load_library().qknorm_rope_strerror(status).decode()


def version() -> int:
    return int(load_library().qknorm_rope_version())


def _check(status: int):
    if status != QKR_OK:
        raise QkrError(status, strerror(status))


def qknorm_rope_fused_raw(qkv: int, q: int, k: int, tokens: int, heads: int, head_dim: int,
                          q_gamma: int, k_gamma: int, eps: float, cos: int, sin: int,
                          cos_layout: int, cos_dtype: int, style: int, dtype: int,
                          stream: int) -> int:
    """The C entry point with integer pointers; returns the raw status."""
    lib = load_library()
    return int(lib.qknorm_rope_fused(qkv or None, q or None, k or None, tokens, heads, head_dim,
                                     q_gamma or None, k_gamma or None, eps, cos or None,
                                     sin or None, cos_layout, cos_dtype, style, dtype,
                                     stream or None))


_torch_module = None
_NO_CONTEXT = contextlib.nullcontext()      # (it may be entered any number of times)


def _torch():
    """torch, imported at the first call that needs it (the raw entry points
    work without)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _x_code(t, names: str = "q/k/qkv") -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return QKR_BF16
    if t.dtype == torch.float16:
        return QKR_FP16
    raise ValueError("%s must be bfloat16 or float16, got %s" % (names, t.dtype))


def _table_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return QKR_FP32
    if t.dtype == torch.bfloat16:
        return QKR_BF16
    raise ValueError("cos/sin must be float32 or bfloat16, got %s" % t.dtype)


def _ptr(t) -> int:
    if t is None:
        return 0
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    return t.data_ptr()


def _current_stream(torch, dev) -> int:
    """The current raw stream of a device.  torch's own raw query saves the
    1.7 us that building a stream object takes."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev.index) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _call_context(ref, tensors, stream):
    """(device context, raw hipStream_t) for a call on ``ref``'s device.

    Every tensor given must live on that device; the call runs with it as the
    current device, so a NULL (default) stream means that device's.
    """
    torch = _torch()
    dev = ref.device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on one device (%s)" % dev)
    if stream is None:
        raw = _current_stream(torch, dev) if ref.is_cuda else 0
    elif isinstance(stream, int):
        raw = stream
    else:
        raw = stream.cuda_stream
    # switching the current device costs a few µs per call: only when needed
    if ref.is_cuda and dev.index != torch.cuda.current_device():
        return torch.cuda.device(dev), raw
    return _NO_CONTEXT, raw


def _launch_stream_context(ref, stream):
    """Context in which tensors the binding allocates for a call belong to the
    stream the call is launched on, so that the caching allocator hands their
    memory to other work only in that stream's order (memory allocated on the
    current stream and freed on return could be reused by the current stream
    while the launch stream still uses it)."""
    if stream is None or not ref.is_cuda:
        return _NO_CONTEXT
    torch = _torch()
    if isinstance(stream, int):
        if stream == torch.cuda.current_stream(ref.device).cuda_stream:
            return _NO_CONTEXT
        stream = torch.cuda.ExternalStream(stream, device=ref.device)
    return torch.cuda.stream(stream)


def qknorm_rope_fused(qkv=None, q=None, k=None, *, q_gamma=None, k_gamma=None,
                      cos=None, sin=None, eps: float = 1e-6, heads: int | None = None,
                      head_dim: int | None = None, cos_layout: str = "shared",
                      style: str = "interleaved", stream=None) -> None:
    """Apply the fused QK-norm + RoPE in place (see ``include/qknorm_rope.h``).

    Fused mode: ``qkv`` is [tokens, 3*heads*head_dim] (any leading shape whose
    last dimension is 3*heads*head_dim); ``head_dim`` defaults to the gamma
    length and ``heads`` to last_dim / (3*head_dim).
    Separate mode: ``q`` and/or ``k`` are [..., heads, head_dim].
    ``cos``/``sin``: [tokens, head_dim] ("shared") or [tokens, heads, head_dim]
    ("per_head"), float32 or bfloat16.  ``stream``: a torch stream or a raw
    hipStream_t integer; defaults to the current stream.
    """
    torch = _torch()
    if qkv is not None:
        ref = qkv
        gam = q_gamma if q_gamma is not None else k_gamma
        if head_dim is None:
            if gam is None:
                raise ValueError("head_dim is needed")
            head_dim = gam.numel()
        if heads is None:
            heads = qkv.shape[-1] // (3 * head_dim)
        if qkv.shape[-1] != 3 * heads * head_dim:
            raise ValueError("qkv last dimension must be 3*heads*head_dim")
        tokens = qkv.numel() // qkv.shape[-1] if qkv.numel() else 0
    else:
        ref = q if q is not None else k
        if ref is None:
            raise ValueError("pass qkv, or q and/or k")
        if ref.dim() < 2:
            raise ValueError("q/k must be [..., heads, head_dim]")
        head_dim = ref.shape[-1] if head_dim is None else head_dim
        heads = ref.shape[-2] if heads is None else heads
        if tuple(ref.shape[-2:]) != (heads, head_dim):
            raise ValueError("q/k must be [..., heads, head_dim] = [..., %d, %d]"
                             % (heads, head_dim))
        tokens = ref.numel() // (heads * head_dim) if ref.numel() else 0
        if q is not None and k is not None and (q.shape != k.shape or q.dtype != k.dtype):
            raise ValueError("q and k must have the same shape and dtype")
    if cos_layout not in LAYOUTS:
        raise ValueError("cos_layout must be one of %s" % sorted(LAYOUTS))
    if style not in STYLES:
        raise ValueError("style must be one of %s" % sorted(STYLES))
    if cos is None or sin is None:
        raise ValueError("cos and sin are required")
    if cos.dtype != sin.dtype or cos.shape != sin.shape:
        raise ValueError("cos and sin must match in shape and dtype")
    rows = tokens * (heads if cos_layout == "per_head" else 1)
    if cos.numel() != rows * head_dim:
        raise ValueError("cos/sin hold %d values, expected %d for the %s layout"
                         % (cos.numel(), rows * head_dim, cos_layout))
    for g in (q_gamma, k_gamma):
        if g is not None and (g.dtype != torch.float32 or g.numel() != head_dim):
            raise ValueError("gamma must be float32 [head_dim]")
    ctx, stream_ptr = _call_context(ref, (qkv, q, k, q_gamma, k_gamma, cos, sin), stream)
    with ctx:
        status = qknorm_rope_fused_raw(
            _ptr(qkv), _ptr(q), _ptr(k), tokens, heads, head_dim, _ptr(q_gamma), _ptr(k_gamma),
            float(eps), _ptr(cos), _ptr(sin), LAYOUTS[cos_layout], _table_code(cos),
            STYLES[style], _x_code(ref), stream_ptr)
    _check(status)


def kernel_info(head_dim: int = 128, cos_layout: str = "shared", cos_dtype: int = QKR_FP32,
                style: str = "interleaved", dtype: int = QKR_BF16, heads: int = 40,
                tokens: int = 32760, tensors: str = "fused") -> dict:
    """Registers, LDS, scratch and schedule of the kernel a call launches.

    ``tensors``: "fused" (one QKV buffer), "pair" (separate q and k) or "one"
    (q or k alone).
    """
    info = KernelInfo()
    _check(load_library().qknorm_rope_kernel_info(head_dim, heads, tokens, TENSORS[tensors],
                                                  LAYOUTS[cos_layout], cos_dtype, STYLES[style],
                                                  dtype, ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in KernelInfo._fields_}


def dit_fuse_scale_shift_raw(x: int, y: int, rows: int, hidden: int, rows_per_batch: int,
                             scale: int, shift: int, mod_dtype: int, eps: float, dtype: int,
                             stream: int) -> int:
    """The AdaLN C entry point with integer pointers; returns the raw status."""
    lib = load_library()
    return int(lib.dit_fuse_scale_shift(x or None, y or None, rows, hidden, rows_per_batch,
                                        scale or None, shift or None, mod_dtype, eps, dtype,
                                        stream or None))


def _mod_code(t, names: str = "scale/shift") -> int:
    torch = _torch()
    dtype = t.dtype
    if dtype == torch.float32:
        return QKR_FP32
    if dtype == torch.bfloat16:
        return QKR_BF16
    if dtype == torch.float16:
        return QKR_FP16
    raise ValueError("%s must be bfloat16, float16 or float32, got %s" % (names, dtype))


def fuse_scale_shift(x, scale, shift, *, out=None, eps: float = 1e-6,
                     rows_per_batch: int | None = None, stream=None):
    """AdaLN modulation (see ``include/fuse_scale_shift.h``); returns ``out``.

    ``x``: [..., hidden] bfloat16/float16; ``scale``/``shift``: [batches, hidden]
    (or [hidden] for one batch) of bfloat16, float16 or float32.  Row r of the
    flattened x uses modulation row r // rows_per_batch; by default the rows
    split evenly over the batches.  ``out`` defaults to a new tensor like x;
    pass ``out=x`` to modulate in place.
    """
    torch = _torch()
    hidden = x.shape[-1]
    rows = x.numel() // hidden if x.numel() else 0
    if scale.shape != shift.shape or scale.dtype != shift.dtype:
        raise ValueError("scale and shift must match in shape and dtype")
    if scale.shape[-1] != hidden:
        raise ValueError("scale/shift last dimension must equal hidden")
    batches = scale.numel() // hidden
    if rows_per_batch is None:
        if batches < 1 or rows % batches:
            raise ValueError("rows do not split evenly over the modulation batches")
        rows_per_batch = max(1, rows // batches)
    if rows and (rows - 1) // rows_per_batch >= batches:
        raise ValueError("scale/shift hold fewer batches than the rows need")
    if out is None:
        with _launch_stream_context(x, stream):
            out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must match x in shape and dtype")
    ctx, stream_ptr = _call_context(x, (out, scale, shift), stream)
    with ctx:
        status = dit_fuse_scale_shift_raw(_ptr(x), _ptr(out), rows, hidden, rows_per_batch,
                                          _ptr(scale), _ptr(shift), _mod_code(scale), float(eps),
                                          _x_code(x, "x"), stream_ptr)
    _check(status)
    return out


def group_norm_silu_workspace_size(n: int, channels: int, spatial: int, groups: int) -> int:
    """Workspace bytes the call needs (negative: a QKR_ERR_* code for bad sizes)."""
    return int(load_library().dit_group_norm_silu_workspace_size(n, channels, spatial, groups))


GN_SCHEDULES = {0: "one_read", 1: "lagged", 2: "two_pass"}


def group_norm_silu_schedule(n: int, channels: int, spatial: int, groups: int):
    """(schedule name, elements per chunk) the library would use for these
    sizes: "one_read", "lagged" or "two_pass" (see include/group_norm_silu.h)."""
    chunk = ctypes.c_int64(0)
    code = int(load_library().dit_group_norm_silu_schedule(n, channels, spatial, groups,
                                                           ctypes.byref(chunk)))
    if code < 0:
        raise QkrError(code, strerror(code))
    return GN_SCHEDULES[code], int(chunk.value)


def dit_group_norm_silu_raw(x: int, y: int, n: int, channels: int, spatial: int, groups: int,
                            gamma: int, beta: int, param_dtype: int, eps: float, dtype: int,
                            workspace: int, workspace_bytes: int, stream: int) -> int:
    """The group-norm C entry point with integer pointers; returns the raw status."""
    lib = load_library()
    return int(lib.dit_group_norm_silu(x or None, y or None, n, channels, spatial, groups,
                                       gamma or None, beta or None, param_dtype, eps, dtype,
                                       workspace or None, workspace_bytes, stream or None))


def dit_group_norm_silu_noalloc_raw(x: int, y: int, n: int, channels: int, spatial: int,
                                    groups: int, gamma: int, beta: int, param_dtype: int,
                                    eps: float, dtype: int, stream: int) -> int:
    """The group-norm entry point that allocates nothing (its workspace is the
    library's fixed per-GPU scratch), with integer pointers; returns the raw
    status."""
    lib = load_library()
    return int(lib.dit_group_norm_silu_noalloc(x or None, y or None, n, channels, spatial, groups,
                                               gamma or None, beta or None, param_dtype, eps,
                                               dtype, stream or None))


def group_norm_silu(x, gamma, beta, groups: int, *, out=None, eps: float = 1e-6,
                    workspace=None, stream=None):
    """Group norm + affine + SiLU (see ``include/group_norm_silu.h``); returns ``out``.

    ``x``: [n, channels, *spatial] bfloat16/float16 (spatial dims flattened,
    their product a multiple of 8).  ``gamma``/``beta``: [channels].
    ``workspace``: a device tensor of at least the queried size; when None and
    one is needed, a byte tensor is allocated here with torch (the library
    itself never allocates), on the launch stream, so its memory is not reused
    before the call's kernels are done with it.  ``out`` defaults to a new
    tensor (also on the launch stream); ``out=x`` works in place.
    """
    torch = _torch()
    if x.dim() < 3:
        raise ValueError("x must be [n, channels, *spatial]")
    n, channels = x.shape[0], x.shape[1]
    spatial = 1
    for d in x.shape[2:]:
        spatial *= d
    if gamma.shape != (channels,) or beta.shape != (channels,) or gamma.dtype != beta.dtype:
        raise ValueError("gamma and beta must be [channels] of one dtype")
    need = group_norm_silu_workspace_size(n, channels, spatial, groups) if x.numel() else 0
    if need < 0:
        raise QkrError(need, strerror(need))
    with _launch_stream_context(x, stream):
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        if out is None:
            out = torch.empty_like(x)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must match x in shape and dtype")
    ctx, stream_ptr = _call_context(x, (out, gamma, beta, workspace), stream)
    with ctx:
        status = dit_group_norm_silu_raw(_ptr(x), _ptr(out), n, channels, spatial, groups,
                                         _ptr(gamma), _ptr(beta), _mod_code(gamma, "gamma/beta"),
                                         float(eps), _x_code(x, "x"), _ptr(workspace), ws_bytes, stream_ptr)
    _check(status)
    return out


def _attn_tensor(t, name: str) -> AttnTensor:
    """t [batch, tokens, heads, head_dim], or without the batch of one sample."""
    strides = t.stride()
    if len(strides) == 3:
        strides = (0, *strides)
    if len(strides) != 4:
        raise ValueError("%s must be [batch, tokens, heads, head_dim]" % name)
    if strides[3] != 1 and t.shape[-1] > 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    return AttnTensor(t.data_ptr(), strides[0], strides[1], strides[2])


def _attn_scale(head_dim: int, scale) -> float:
    if scale is not None:
        return scale
    return head_dim ** -0.5 if head_dim else 1.0       # (no head_dim: the library refuses the call)


def _attn_args(q, k, v, causal, kv_lengths, scale) -> AttnArgs:
    torch = _torch()
    shape, kv_shape = q.shape, k.shape
    if len(shape) == 3:
        shape = (1, *shape)
        kv_shape = (1, *kv_shape)
    if len(shape) != 4 or len(kv_shape) != 4:
        raise ValueError("q, k and v must be [batch, tokens, heads, head_dim]")
    batch, q_tokens, heads, head_dim = shape
    if k.shape != v.shape or kv_shape[0] != batch or kv_shape[3] != head_dim:
        raise ValueError("k and v must be [%d, kv_tokens, kv_heads, %d]" % (batch, head_dim))
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one dtype")
    kv_heads = kv_shape[2]
    if kv_heads < 1 or heads % kv_heads:
        raise ValueError("the number of query heads must be a multiple of k's and v's")
    if kv_lengths is not None and (kv_lengths.dtype != torch.int32 or kv_lengths.shape != (batch,)):
        raise ValueError("kv_lengths must be int32 [batch]")
    return AttnArgs(batch, q_tokens, kv_shape[1], heads, kv_heads, head_dim, 1 if causal else 0,
                    _x_code(q, "q/k/v"), _attn_scale(head_dim, scale),
                    None if kv_lengths is None else _ptr(kv_lengths))


def _lse_shape(q):
    return (*q.shape[:-3], q.shape[-2], q.shape[-3])


def _check_lse(lse, q):
    if tuple(lse.shape) != _lse_shape(q) or lse.dtype != _torch().float32:
        raise ValueError("lse must be float32 [batch, heads, tokens]")


def _attn_workspace(size_of, args, workspace, device):
    """(workspace, its bytes), allocated here if the call needs one and has none."""
    if workspace is None:
        need = int(size_of(ctypes.byref(args)))
        if need < 0:
            raise QkrError(need, strerror(need))
        if need > 0:
            workspace = _torch().empty(need, dtype=_torch().uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size() if workspace is not None else 0


def attention_workspace_size(batch: int, q_tokens: int, kv_tokens: int, heads: int, kv_heads: int,
                             head_dim: int, *, causal: bool = False, dtype: int = QKR_BF16,
                             backward: bool = False) -> int:
    """Workspace bytes of an attention call, or of its backward pass (negative:
    a QKR_ERR_* code for bad sizes)."""
    lib = load_library()
    args = AttnArgs(batch, q_tokens, kv_tokens, heads, kv_heads, head_dim, 1 if causal else 0, dtype,
                    1.0, None)
    size_of = lib.dit_attention_backward_workspace_size if backward else lib.dit_attention_workspace_size
    return int(size_of(ctypes.byref(args)))


def attention(q, k, v, *, causal: bool = False, kv_lengths=None, scale: float | None = None,
              out=None, lse=None, workspace=None, stream=None):
    """Attention (see ``include/dit_attention.h``); returns ``(out, lse)``.

    ``q``: [batch, tokens, heads, head_dim], ``k``/``v``: [batch, kv_tokens,
    kv_heads, head_dim] of bfloat16 or float16 (or without the batch dimension
    for one sample); any strides that are multiples of 8 with the last
    dimension contiguous, so the slices of a fused QKV buffer serve as they
    are (a dimension of one element may have any stride).  ``heads`` is a
    multiple of ``kv_heads``; consecutive query heads share a key head.
    ``kv_lengths``: int32 [batch], the keys in use of each sample.
    ``causal``: the last query sees the last key of kv_tokens, the one before
    it one key fewer.  ``scale`` defaults to head_dim ** -0.5.
    ``out`` (like q, same rules for strides) and ``lse`` (float32 [batch,
    heads, tokens], the log of each row's sum of exponentials, which the
    backward pass takes) default to new tensors.  ``workspace``: a device
    tensor of at least ``attention_workspace_size`` bytes; allocated here on
    the launch stream when None and one is needed.
    """
    torch = _torch()
    lib = load_library()
    args = _attn_args(q, k, v, causal, kv_lengths, scale)
    with _launch_stream_context(q, stream):
        workspace, ws_bytes = _attn_workspace(lib.dit_attention_workspace_size, args, workspace,
                                              q.device)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty(_lse_shape(q), dtype=torch.float32, device=q.device)
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q in shape and dtype")
    _check_lse(lse, q)
    ctx, stream_ptr = _call_context(q, (k, v, out, lse, kv_lengths, workspace), stream)
    with ctx:
        status = lib.dit_attention(args, _attn_tensor(q, "q"), _attn_tensor(k, "k"),
                                   _attn_tensor(v, "v"), _attn_tensor(out, "out"), _ptr(lse),
                                   _ptr(workspace), ws_bytes, stream_ptr)
    _check(status)
    return out, lse


def attention_backward(dout, q, k, v, out, lse, *, causal: bool = False, kv_lengths=None,
                       scale: float | None = None, dq=None, dk=None, dv=None, workspace=None,
                       stream=None):
    """Backward pass of ``attention``; returns ``(dq, dk, dv)``.

    ``dout`` is the gradient of ``out``; ``q``, ``k``, ``v``, ``out``, ``lse``
    and the masks are the forward call's.  ``dq``, ``dk`` and ``dv`` are
    written (not added to) and default to new contiguous tensors; they may be
    the slices of one fused gradient buffer.  Tensors follow the forward
    call's rules; a dout without its own memory for every token (an expanded
    one) has to be made contiguous first.
    """
    torch = _torch()
    lib = load_library()
    args = _attn_args(q, k, v, causal, kv_lengths, scale)
    with _launch_stream_context(q, stream):
        workspace, ws_bytes = _attn_workspace(lib.dit_attention_backward_workspace_size, args,
                                              workspace, q.device)
        if dq is None:
            dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if dk is None:
            dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        if dv is None:
            dv = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    for name, t, like in (("dout", dout, q), ("out", out, q), ("dq", dq, q), ("dk", dk, k),
                          ("dv", dv, v)):
        if t.shape != like.shape or t.dtype != like.dtype:
            raise ValueError("%s must match %s in shape and dtype"
                             % (name, {"dk": "k", "dv": "v"}.get(name, "q")))
    _check_lse(lse, q)
    ctx, stream_ptr = _call_context(q, (dout, k, v, out, lse, dq, dk, dv, kv_lengths, workspace),
                                    stream)
    with ctx:
        status = lib.dit_attention_backward(
            args, _attn_tensor(dout, "dout"), _attn_tensor(q, "q"), _attn_tensor(k, "k"),
            _attn_tensor(v, "v"), _attn_tensor(out, "out"), _ptr(lse), _attn_tensor(dq, "dq"),
            _attn_tensor(dk, "dk"), _attn_tensor(dv, "dv"), _ptr(workspace), ws_bytes, stream_ptr)
    _check(status)
    return dq, dk, dv


def _small(what: str, *sizes):
    """Sizes that the C interface takes in 32 bits: ctypes would cut larger ones off."""
    if max(sizes) > 0x7fffffff:
        raise ValueError("%s must be below 2^31" % what)


def _packed_args(q, k, v, offsets, kv_offsets, causal, scale, fill) -> AttnPackedArgs:
    torch = _torch()
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, head_dim]")
    q_tokens, heads, head_dim = q.shape
    if k.shape != v.shape or k.shape[2] != head_dim:
        raise ValueError("k and v must be [kv_tokens, kv_heads, %d]" % head_dim)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one dtype")
    kv_heads = k.shape[1]
    if kv_heads < 1 or heads % kv_heads:
        raise ValueError("the number of query heads must be a multiple of k's and v's")
    _small("heads and head_dim", heads, head_dim)
    if kv_offsets is None and k.shape[0] != q_tokens:
        raise ValueError("k and v of other tokens than q need kv_offsets")
    if offsets.dim() != 1 or offsets.numel() < 1 or offsets.dtype != torch.int32:
        raise ValueError("offsets must be int32 [sequences + 1]")
    if kv_offsets is not None and (kv_offsets.shape != offsets.shape or kv_offsets.dtype != torch.int32):
        raise ValueError("kv_offsets must be int32 [sequences + 1], as offsets are")
    return AttnPackedArgs(offsets.numel() - 1, q_tokens, k.shape[0], heads, kv_heads, head_dim,
                          1 if causal else 0, _x_code(q, "q/k/v"),
                          _attn_scale(head_dim, scale), 1 if fill else 0, _ptr(offsets),
                          None if kv_offsets is None else _ptr(kv_offsets))


def attention_packed_workspace_size(sequences: int, q_tokens: int, kv_tokens: int, heads: int, kv_heads: int,
                                    head_dim: int, *, causal: bool = False, dtype: int = QKR_BF16,
                                    backward: bool = False) -> int:
    """Workspace bytes of an ``attention_packed`` call of buffers of these rows,
    or of its backward pass (negative: a QKR_ERR_* code for bad sizes)."""
    lib = load_library()
    args = AttnPackedArgs(sequences, q_tokens, kv_tokens, heads, kv_heads, head_dim, 1 if causal else 0, dtype,
                          1.0, 0, None, None)
    size_of = (lib.dit_attention_packed_backward_workspace_size if backward
               else lib.dit_attention_packed_workspace_size)
    return int(size_of(args))


def attention_packed(q, k, v, offsets, *, kv_offsets=None, causal: bool = False, scale: float | None = None,
                     out=None, lse=None, workspace=None, stream=None):
    """Attention of packed sequences of different lengths (see
    ``include/dit_attention.h``); returns ``(out, lse)``.

    ``q``: [tokens, heads, head_dim], ``k``/``v``: [kv_tokens, kv_heads,
    head_dim], sequences one after another, of the types and strides that
    ``attention`` takes.  ``offsets``: int32 [sequences + 1] on the GPU, not
    decreasing: sequence i has the rows offsets[i] to offsets[i + 1] - 1 of q,
    and of k and v unless ``kv_offsets`` (like it) says which.  Each attends to
    its own keys as a sample of ``attention`` does; ``causal``: its last query
    sees its last key.  Rows of no sequence, before the first or behind the
    last, count for nothing, whatever they hold, and are left as they are in
    ``out`` and ``lse`` (float32 [heads, tokens]); where both are made here, they
    hold 0 and -inf there.
    ``workspace``: at least ``attention_packed_workspace_size`` bytes, allocated
    here on the launch stream when None and one is needed.
    """
    torch = _torch()
    lib = load_library()
    args = _packed_args(q, k, v, offsets, kv_offsets, causal, scale, out is None and lse is None)
    with _launch_stream_context(q, stream):
        workspace, ws_bytes = _attn_workspace(lib.dit_attention_packed_workspace_size, args, workspace,
                                              q.device)
        if out is None:
            out = (q.new_empty if args.fill_rest else q.new_zeros)(q.shape)
        if lse is None:
            lse = q.new_empty(_lse_shape(q), dtype=torch.float32)
            if not args.fill_rest:
                lse.fill_(-float("inf"))
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q in shape and dtype")
    _check_lse(lse, q)
    ctx, stream_ptr = _call_context(q, (k, v, out, lse, offsets, kv_offsets, workspace), stream)
    with ctx:
        status = lib.dit_attention_packed(args, _attn_tensor(q, "q"), _attn_tensor(k, "k"),
                                          _attn_tensor(v, "v"), _attn_tensor(out, "out"), _ptr(lse),
                                          _ptr(workspace), ws_bytes, stream_ptr)
    _check(status)
    return out, lse


def attention_packed_backward(dout, q, k, v, out, lse, offsets, *, kv_offsets=None, causal: bool = False,
                              scale: float | None = None, dq=None, dk=None, dv=None, workspace=None,
                              stream=None):
    """Backward pass of ``attention_packed``; returns ``(dq, dk, dv)``.

    The arguments are those of the forward call and of ``attention_backward``.
    Rows of no sequence are left as they are in gradients that are given, and 0
    in those made here.
    """
    lib = load_library()
    args = _packed_args(q, k, v, offsets, kv_offsets, causal, scale, dq is None and dk is None and dv is None)
    make = q.new_empty if args.fill_rest else q.new_zeros
    with _launch_stream_context(q, stream):
        workspace, ws_bytes = _attn_workspace(lib.dit_attention_packed_backward_workspace_size, args,
                                              workspace, q.device)
        if dq is None:
            dq = make(q.shape)
        if dk is None:
            dk = make(k.shape)
        if dv is None:
            dv = make(v.shape)
    for name, t, like in (("dout", dout, q), ("out", out, q), ("dq", dq, q), ("dk", dk, k),
                          ("dv", dv, v)):
        if t.shape != like.shape or t.dtype != like.dtype:
            raise ValueError("%s must match %s in shape and dtype"
                             % (name, {"dk": "k", "dv": "v"}.get(name, "q")))
    _check_lse(lse, q)
    ctx, stream_ptr = _call_context(q, (dout, k, v, out, lse, dq, dk, dv, offsets, kv_offsets, workspace),
                                    stream)
    with ctx:
        status = lib.dit_attention_packed_backward(
            args, _attn_tensor(dout, "dout"), _attn_tensor(q, "q"), _attn_tensor(k, "k"),
            _attn_tensor(v, "v"), _attn_tensor(out, "out"), _ptr(lse), _attn_tensor(dq, "dq"),
            _attn_tensor(dk, "dk"), _attn_tensor(dv, "dv"), _ptr(workspace), ws_bytes, stream_ptr)
    _check(status)
    return dq, dk, dv


def layer_norm(x, weight=None, bias=None, *, out=None, eps: float = 1e-6, stream=None):
    """Layer norm over the last dimension (see ``include/layer_norm.h``); returns ``out``.

    ``x``: [..., hidden] bfloat16/float16; ``weight``/``bias``: [hidden] of one
    of bfloat16, float16 or float32, either may be None.  ``out`` defaults to
    a new tensor like x; pass ``out=x`` to normalise in place.
    """
    torch = _torch()
    hidden = x.shape[-1]
    rows = x.numel() // hidden if x.numel() else 0
    for p in (weight, bias):
        if p is not None and p.shape != (hidden,):
            raise ValueError("weight and bias must be [%d]" % hidden)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one dtype")
    one = weight if weight is not None else bias
    if out is None:
        with _launch_stream_context(x, stream):
            out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must match x in shape and dtype")
    ctx, stream_ptr = _call_context(x, (out, weight, bias), stream)
    with ctx:
        status = load_library().dit_layer_norm(
            _ptr(x), _ptr(out), rows, hidden, _ptr(weight),
            _ptr(bias), QKR_FP32 if one is None else _mod_code(one, "weight/bias"), float(eps),
            _x_code(x, "x"), stream_ptr)
    _check(status)
    return out


def layer_norm_backward_workspace_size(rows: int, hidden: int, rows_per_batch: int | None = None) -> int:
    """Workspace bytes of ``layer_norm_backward`` (or, with rows_per_batch, of
    ``fuse_scale_shift_backward``); negative: a QKR_ERR_* code."""
    return int(load_library().dit_layer_norm_backward_workspace_size(
        rows, hidden, max(1, rows) if rows_per_batch is None else rows_per_batch))


def _norm_backward(dy, x, weight, form, rows, hidden, rows_per_batch, params_shape, out, eps,
                   workspace, stream):
    torch = _torch()
    lib = load_library()
    device = x.device
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must match x in shape and dtype")
    if out is not None and (out.shape != x.shape or out.dtype != x.dtype):
        raise ValueError("out must match x in shape and dtype")
    dweight = dbias = None
    ws_bytes = 0
    with _launch_stream_context(x, stream):
        if params_shape is not None:
            make = torch.empty if rows else torch.zeros     # without rows the sums are empty
            dweight = make(params_shape, dtype=torch.float32, device=device)
            dbias = make(params_shape, dtype=torch.float32, device=device)
            if workspace is None:
                ws_bytes = lib.dit_layer_norm_backward_workspace_size(rows, hidden, rows_per_batch)
                if ws_bytes < 0:
                    raise QkrError(ws_bytes, strerror(ws_bytes))
                if ws_bytes > 0:
                    workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
            else:
                ws_bytes = workspace.numel() * workspace.element_size()
        if out is None:
            out = torch.empty_like(x)
    ctx, stream_ptr = _call_context(x, (dy, out, weight, workspace), stream)
    with ctx:
        status = lib.dit_layer_norm_backward(
            _ptr(dy), _ptr(x), _ptr(out), rows, hidden, rows_per_batch, _ptr(weight), form,
            QKR_FP32 if weight is None else _mod_code(weight, "scale" if form else "weight"),
            _ptr(dweight), _ptr(dbias), float(eps), _x_code(x, "x"), _ptr(workspace), ws_bytes, stream_ptr)
    _check(status)
    return out, dweight, dbias


def layer_norm_backward(dy, x, weight=None, *, out=None, eps: float = 1e-6,
                        param_grads: bool | None = None, workspace=None, stream=None):
    """Backward pass of ``layer_norm``; returns ``(dx, dweight, dbias)``.

    ``dy``: the gradient of its output, ``x``: its input.  ``dweight`` and
    ``dbias`` are float32 [hidden], or None without ``param_grads``, which
    defaults to whether there is a ``weight``: pass True for the gradient of a
    bias alone, False where the weight gets none.
    ``out`` receives dx (a new tensor by default); ``out=dy`` works in place.
    ``workspace``: at least ``layer_norm_backward_workspace_size`` bytes;
    allocated here on the launch stream when None and needed.
    """
    hidden = x.shape[-1]
    if weight is not None and weight.shape != (hidden,):
        raise ValueError("weight must be [%d]" % hidden)
    rows = x.numel() // hidden if hidden else 0
    if param_grads is None:
        param_grads = weight is not None
    return _norm_backward(dy, x, weight, DIT_LN_WEIGHT, rows, hidden, max(1, rows),
                          hidden if param_grads else None, out, eps, workspace, stream)


def fuse_scale_shift_backward(dy, x, scale, *, out=None, eps: float = 1e-6,
                              rows_per_batch: int | None = None, workspace=None, stream=None):
    """Backward pass of ``fuse_scale_shift``; returns ``(dx, dscale, dshift)``.

    ``dy``: the gradient of its output; ``x``, ``scale`` and
    ``rows_per_batch``: the forward call's.  ``dscale`` and ``dshift`` are
    float32 in scale's shape, each row summed over the rows of x that use it
    (zero where none does).  ``out`` and ``workspace``: as in
    ``layer_norm_backward``.
    """
    hidden = x.shape[-1]
    rows = x.numel() // hidden if x.numel() else 0
    if scale.shape[-1] != hidden:
        raise ValueError("scale's last dimension must equal hidden")
    batches = scale.numel() // hidden
    if rows_per_batch is None:
        if batches < 1 or rows % batches:
            raise ValueError("rows do not split evenly over the modulation batches")
        rows_per_batch = max(1, rows // batches)
    used = -(-rows // rows_per_batch) if rows_per_batch > 0 else 0
    if used > batches:
        raise ValueError("scale holds fewer batches than the rows need")
    dx, dscale, dshift = _norm_backward(dy, x, scale, DIT_LN_ONE_PLUS, rows, hidden, rows_per_batch,
                                        scale.shape, out, eps, workspace, stream)
    if 0 < used < batches:
        with _launch_stream_context(x, stream):
            for t in (dscale, dshift):
                t.view(batches, hidden)[used:].zero_()
    return dx, dscale, dshift


def _like(t, x, name: str, like: str = "x"):
    if t.shape != x.shape or t.dtype != x.dtype:
        raise ValueError("%s must match %s in shape and dtype" % (name, like))


def _rms_norm(x, weight, residual, sum_out, out, scales, eps, stream):
    lib = load_library()
    rows = x.numel() // x.shape[-1] if x.numel() else 0
    ctx, stream_ptr = _call_context(x, (residual, sum_out, out, scales, weight), stream)
    with ctx:
        status = lib.dit_rms_norm(
            _ptr(x), _ptr(residual), _ptr(sum_out), _ptr(out), _ptr(scales), rows, x.shape[-1],
            _ptr(weight), QKR_FP32 if weight is None else _mod_code(weight, "weight"), float(eps),
            _x_code(x, "x"), stream_ptr)
    _check(status)


def _rms_norm_sum(x, weight, residual, sum_out):
    """The checks that both forms share; sum_out, made here if there is a residual."""
    if x.dim() < 1:
        raise ValueError("x must be [..., hidden]")
    _small("hidden", x.shape[-1])
    if weight is not None and weight.shape != x.shape[-1:]:
        raise ValueError("weight must be [%d]" % x.shape[-1])
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out needs a residual")
        return None
    _like(residual, x, "residual")
    if sum_out is None:
        return _torch().empty_like(x)
    _like(sum_out, x, "sum_out")
    return sum_out


def rms_norm(x, weight=None, *, residual=None, sum_out=None, out=None, eps: float = 1e-6, stream=None):
    """RMS norm over the last dimension (see ``include/rms_norm.h``); returns
    ``out``, or ``(out, sum)`` with a residual.

    ``x``: [..., hidden] bfloat16/float16; ``weight``: [hidden] of bfloat16,
    float16 or float32, or None.  ``residual``, like x, is added first: the sum
    is rounded to x's type, is what is normalised, and goes to ``sum_out`` (a
    new tensor by default; ``sum_out=residual`` adds in place).  ``out``
    defaults to a new tensor like x; it may be x or the residual itself.
    """
    with _launch_stream_context(x, stream):
        sum_out = _rms_norm_sum(x, weight, residual, sum_out)
        if out is None:
            out = _torch().empty_like(x)
        else:
            _like(out, x, "out")
    _rms_norm(x, weight, residual, sum_out, out, None, eps, stream)
    return out if residual is None else (out, sum_out)


def rms_norm_fp8(x, weight=None, *, residual=None, sum_out=None, out=None, scales=None,
                 eps: float = 1e-6, stream=None):
    """``rms_norm`` with an output in 8 bits; returns ``(out, scales)``, or
    ``(out, scales, sum)`` with a residual.

    ``out`` is float8_e4m3fn in x's shape, ``scales`` float32 in x's shape
    without its last dimension: a row's largest value becomes 448, and the norm
    is ``out * scales`` of the row (0 * anything for a row of zeros).  They are
    what ``gated_feed_forward`` takes as ``x`` and ``x_scale``.  The other
    arguments are ``rms_norm``'s.
    """
    torch = _torch()
    with _launch_stream_context(x, stream):
        sum_out = _rms_norm_sum(x, weight, residual, sum_out)
        if out is None:
            # (contiguous whatever x's strides are; empty_like is half of empty's 2.3 us)
            out = torch.empty_like(x, dtype=torch.float8_e4m3fn, memory_format=torch.contiguous_format)
        elif out.shape != x.shape or out.dtype != torch.float8_e4m3fn:
            raise ValueError("out must be float8_e4m3fn in x's shape")
        if scales is None:
            scales = x.new_empty(x.shape[:-1], dtype=torch.float32)
        elif scales.shape != x.shape[:-1] or scales.dtype != torch.float32:
            raise ValueError("scales must be float32, one a row of x")
    _rms_norm(x, weight, residual, sum_out, out, scales, eps, stream)
    return (out, scales) if residual is None else (out, scales, sum_out)


def rms_norm_backward_workspace_size(rows: int, hidden: int) -> int:
    """Workspace bytes of ``rms_norm_backward`` (negative: a QKR_ERR_* code)."""
    return int(load_library().dit_rms_norm_backward_workspace_size(rows, hidden))


def rms_norm_backward(dy, x, weight=None, *, dsum=None, out=None, eps: float = 1e-6,
                      param_grads: bool | None = None, workspace=None, stream=None):
    """Backward pass of ``rms_norm``; returns ``(dx, dweight)``.

    ``dy``: the gradient of its output, ``x``: what it normalised (the sum, if
    there was a residual).  ``dsum``, like x, is the gradient that reaches the
    sum past the norm, and is added: dx is then the gradient of x and of the
    residual alike.  ``dweight`` is float32 [hidden], or None without
    ``param_grads``, which defaults to whether there is a ``weight``.
    ``out`` receives dx (a new tensor by default); it may be dy or dsum itself.
    ``workspace``: at least ``rms_norm_backward_workspace_size`` bytes;
    allocated here on the launch stream when None and needed.
    """
    torch = _torch()
    lib = load_library()
    if x.dim() < 1:
        raise ValueError("x must be [..., hidden]")
    hidden = x.shape[-1]
    _small("hidden", hidden)
    rows = x.numel() // hidden if x.numel() else 0
    if weight is not None and weight.shape != (hidden,):
        raise ValueError("weight must be [%d]" % hidden)
    for name, t in (("dy", dy), ("dsum", dsum), ("out", out)):
        if t is not None:
            _like(t, x, name)
    if param_grads is None:
        param_grads = weight is not None
    dweight = None
    ws_bytes = 0
    with _launch_stream_context(x, stream):
        if param_grads:
            make = x.new_empty if rows else x.new_zeros     # without rows the sum is empty
            dweight = make(hidden, dtype=torch.float32)
            if workspace is None:
                ws_bytes = lib.dit_rms_norm_backward_workspace_size(rows, hidden)
                if ws_bytes < 0:
                    raise QkrError(ws_bytes, strerror(ws_bytes))
                if ws_bytes > 0:
                    workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
            else:
                ws_bytes = workspace.numel() * workspace.element_size()
        if out is None:
            out = torch.empty_like(x)
    ctx, stream_ptr = _call_context(x, (dy, dsum, out, weight, workspace), stream)
    with ctx:
        status = lib.dit_rms_norm_backward(
            _ptr(dy), _ptr(x), _ptr(dsum), _ptr(out), rows, hidden, _ptr(weight),
            QKR_FP32 if weight is None else _mod_code(weight, "weight"), _ptr(dweight), float(eps),
            _x_code(x, "x"), _ptr(workspace), ws_bytes, stream_ptr)
    _check(status)
    return out, dweight


def qknorm_rope_backward_workspace_size(tokens: int, head_dim: int) -> int:
    """Workspace bytes the call needs (negative: a QKR_ERR_* code for bad sizes)."""
    return int(load_library().qknorm_rope_backward_workspace_size(tokens, head_dim))


def qknorm_rope_backward(dqkv=None, qkv=None, dq=None, dk=None, q=None, k=None, *, q_gamma=None,
                         k_gamma=None, cos=None, sin=None, eps: float = 1e-6,
                         heads: int | None = None, head_dim: int | None = None,
                         cos_layout: str = "shared", style: str = "interleaved", out=None,
                         dq_out=None, dk_out=None, workspace=None, stream=None):
    """Backward pass of ``qknorm_rope_fused`` (see ``include/qknorm_rope_backward.h``);
    returns ``(dq_gamma, dk_gamma)``, float32 [head_dim], and writes dx.

    Fused mode: ``dqkv`` holds the gradients of the pass's output in its Q and
    K slices, ``qkv`` the pass's input (a copy taken before the pass wrote
    over it).  dx replaces the Q and K slices of ``dqkv``, or goes to those of
    ``out``; V slices are neither read nor written.
    Separate mode: ``dq`` with ``q`` and/or ``dk`` with ``k``, [..., heads,
    head_dim]; dx replaces dq and dk, or goes to ``dq_out`` and ``dk_out``.
    The gradient of a weight whose tensor is not given is None.  The other
    arguments are the forward call's; ``workspace``: at least
    ``qknorm_rope_backward_workspace_size`` bytes, allocated here on the launch
    stream when None.
    """
    torch = _torch()
    lib = load_library()
    if dqkv is not None:
        if qkv is None or any(t is not None for t in (dq, dk, q, k)):
            raise ValueError("pass dqkv with qkv, or dq with q and/or dk with k")
        ref = qkv
        gam = q_gamma if q_gamma is not None else k_gamma
        if head_dim is None:
            if gam is None:
                raise ValueError("head_dim is needed")
            head_dim = gam.numel()
        if heads is None:
            heads = qkv.shape[-1] // (3 * head_dim)
        if qkv.shape[-1] != 3 * heads * head_dim:
            raise ValueError("qkv last dimension must be 3*heads*head_dim")
        tokens = qkv.numel() // qkv.shape[-1] if qkv.numel() else 0
        tensors = (dqkv, qkv, dqkv if out is None else out)
        fused = GradTensor(_ptr(dqkv), _ptr(qkv), _ptr(tensors[2]))
        of_q = of_k = None
    else:
        if qkv is not None or (dq is None) != (q is None) or (dk is None) != (k is None) \
                or (q is None and k is None):
            raise ValueError("pass dqkv with qkv, or dq with q and/or dk with k")
        ref = q if q is not None else k
        if ref.dim() < 2:
            raise ValueError("q/k must be [..., heads, head_dim]")
        head_dim = ref.shape[-1] if head_dim is None else head_dim
        heads = ref.shape[-2] if heads is None else heads
        if tuple(ref.shape[-2:]) != (heads, head_dim):
            raise ValueError("q/k must be [..., heads, head_dim] = [..., %d, %d]"
                             % (heads, head_dim))
        tokens = ref.numel() // (heads * head_dim) if ref.numel() else 0
        fused = of_q = of_k = None
        tensors = ()
        if q is not None:
            tensors = (dq, q, dq if dq_out is None else dq_out)
            of_q = GradTensor(*map(_ptr, tensors))
        if k is not None:
            more = (dk, k, dk if dk_out is None else dk_out)
            of_k = GradTensor(*map(_ptr, more))
            tensors += more
    shape, dtype = ref.shape, ref.dtype
    for t in tensors:
        if t.shape != shape or t.dtype != dtype:
            raise ValueError("gradients, inputs and outputs must have one shape and dtype")
    if cos_layout not in LAYOUTS:
        raise ValueError("cos_layout must be one of %s" % sorted(LAYOUTS))
    if style not in STYLES:
        raise ValueError("style must be one of %s" % sorted(STYLES))
    if cos is None or sin is None:
        raise ValueError("cos and sin are required")
    if cos.dtype != sin.dtype or cos.shape != sin.shape:
        raise ValueError("cos and sin must match in shape and dtype")
    rows = tokens * (heads if cos_layout == "per_head" else 1)
    if cos.numel() != rows * head_dim:
        raise ValueError("cos/sin hold %d values, expected %d for the %s layout"
                         % (cos.numel(), rows * head_dim, cos_layout))
    for g in (q_gamma, k_gamma):
        if g is not None and (g.dtype != torch.float32 or g.numel() != head_dim):
            raise ValueError("gamma must be float32 [head_dim]")
    with _launch_stream_context(ref, stream):
        dq_gamma = dk_gamma = None
        if of_k is None or of_q is not None:
            dq_gamma = torch.empty(head_dim, dtype=torch.float32, device=ref.device)
        if of_q is None or of_k is not None:
            dk_gamma = torch.empty(head_dim, dtype=torch.float32, device=ref.device)
        if workspace is None:
            need = qknorm_rope_backward_workspace_size(tokens, head_dim)
            if need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=ref.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    ctx, stream_ptr = _call_context(ref, (*tensors, q_gamma, k_gamma, cos, sin, workspace), stream)
    with ctx:
        status = lib.qknorm_rope_backward(
            fused, of_q, of_k, tokens, heads, head_dim, _ptr(q_gamma), _ptr(k_gamma),
            _ptr(dq_gamma), _ptr(dk_gamma), float(eps), _ptr(cos), _ptr(sin), LAYOUTS[cos_layout],
            _table_code(cos), STYLES[style], _x_code(ref), _ptr(workspace), ws_bytes, stream_ptr)
    _check(status)
    return dq_gamma, dk_gamma


def _ff_args(x, w_gate, w_up, activation, out_dtype=None) -> FfArgs:
    torch = _torch()
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be one of %s" % sorted(ACTIVATIONS))
    if x.dim() < 1 or w_gate.dim() != 2 or w_gate.shape[1] != x.shape[-1]:
        raise ValueError("x must be [..., hidden] and the weights [inner, hidden]")
    if w_up.shape != w_gate.shape:
        raise ValueError("w_gate and w_up must have one shape")
    if w_gate.dtype != x.dtype or w_up.dtype != x.dtype:
        raise ValueError("x, w_gate and w_up must have one dtype")
    inner, hidden = w_gate.shape
    _small("hidden and inner", hidden, inner)
    if x.dtype == torch.float8_e4m3fn:
        dtype = DIT_FF_E4M3
        out = {None: QKR_BF16, torch.bfloat16: QKR_BF16, torch.float16: QKR_FP16}.get(out_dtype)
        if out is None:
            raise ValueError("out_dtype must be bfloat16 or float16, got %s" % out_dtype)
    else:
        dtype = out = _x_code(x, "x and the weights")
        if out_dtype is not None and out_dtype != x.dtype:
            raise ValueError("out_dtype must be x's dtype, unless that is float8_e4m3fn")
    return FfArgs(x.numel() // hidden if hidden else 0, hidden, inner, ACTIVATIONS[activation], dtype, out)


def _ff_like(t, shape, dtype, name: str):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError("%s must be %s %s" % (name, dtype, list(shape)))


def gated_feed_forward(x, w_gate, w_up, *, activation: str = "silu", x_scale=None, gate_scale=None,
                       up_scale=None, out_dtype=None, save: bool = False, out=None, gate=None,
                       up=None, stream=None):
    """``act(x @ w_gate.T) * (x @ w_up.T)`` in one kernel (see
    ``include/feed_forward.h``); returns ``out``, or ``(out, gate, up)`` with
    ``save``.

    ``x``: [..., hidden]; ``w_gate``/``w_up``: [inner, hidden] (the halves of
    one [2 * inner, hidden] weight serve as they are), all of bfloat16 or
    float16, or all of float8_e4m3fn with ``x_scale`` (float32, one a row of x:
    what ``rms_norm_fp8`` gives) and ``gate_scale``/``up_scale`` (float32
    [inner]).  ``activation``: "silu" or "gelu_tanh".  ``out``: [..., inner] of
    x's dtype, or for 8 bits of ``out_dtype`` (bfloat16 by default).  ``save``
    keeps both projections in ``gate`` and ``up``, like out, for
    ``gated_feed_forward_backward``.
    """
    torch = _torch()
    lib = load_library()
    args = _ff_args(x, w_gate, w_up, activation, out_dtype)
    fp8 = args.dtype == DIT_FF_E4M3
    for name, t, shape in (("x_scale", x_scale, x.shape[:-1]), ("gate_scale", gate_scale, (args.inner,)),
                           ("up_scale", up_scale, (args.inner,))):
        if fp8 != (t is not None):
            raise ValueError("%s goes with float8_e4m3fn, and only with it" % name)
        if t is not None:
            _ff_like(t, shape, torch.float32, name)
    if not save and (gate is not None or up is not None):
        raise ValueError("gate and up go with save")
    shape = (*x.shape[:-1], args.inner)
    dtype = torch.float16 if args.out_dtype == QKR_FP16 else torch.bfloat16
    made = []
    with _launch_stream_context(x, stream):
        for name, t, wanted in (("out", out, True), ("gate", gate, save), ("up", up, save)):
            if t is not None:
                _ff_like(t, shape, dtype, name)
            elif wanted:
                t = x.new_empty(shape, dtype=dtype)
            made.append(t)
    out, gate, up = made
    ctx, stream_ptr = _call_context(x, (w_gate, w_up, x_scale, gate_scale, up_scale, out, gate, up), stream)
    with ctx:
        status = lib.dit_gated_feed_forward(args, _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(x_scale),
                                            _ptr(gate_scale), _ptr(up_scale), _ptr(out), _ptr(gate), _ptr(up),
                                            stream_ptr)
    _check(status)
    return (out, gate, up) if save else out


def gated_feed_forward_backward_workspace_size(rows: int, hidden: int, inner: int, *,
                                               dtype: int = QKR_BF16) -> int:
    """Workspace bytes of ``gated_feed_forward_backward`` (negative: a QKR_ERR_*
    code for bad sizes)."""
    args = FfArgs(rows, hidden, inner, 0, dtype, dtype)
    return int(load_library().dit_gated_feed_forward_backward_workspace_size(args))


def gated_feed_forward_backward(dh, x, w_gate, w_up, gate, up, *, activation: str = "silu", dx=None,
                                dw_gate=None, dw_up=None, input_grad: bool = True,
                                weight_grads: bool = True, workspace=None, stream=None):
    """Backward pass of ``gated_feed_forward``; returns ``(dx, dw_gate, dw_up)``.

    ``dh`` is the gradient of its output, ``gate`` and ``up`` what it saved; the
    rest is the forward call's, of bfloat16 or float16.  Gradients are of that
    dtype, written (not added to), and default to new tensors; dx is None
    without ``input_grad``, the other two are without ``weight_grads``.
    ``workspace``: at least ``gated_feed_forward_backward_workspace_size`` bytes
    (4 bytes an element of dh, more for few rows); allocated here on the launch
    stream when None.
    """
    torch = _torch()
    lib = load_library()
    args = _ff_args(x, w_gate, w_up, activation)
    if args.dtype == DIT_FF_E4M3:
        raise ValueError("the backward pass takes bfloat16 or float16")
    shape = (*x.shape[:-1], args.inner)
    for name, t in (("dh", dh), ("gate", gate), ("up", up)):
        _ff_like(t, shape, x.dtype, name)
    for name, t, wanted in (("dx", dx, input_grad), ("dw_gate", dw_gate, weight_grads), ("dw_up", dw_up, weight_grads)):
        if t is not None and not wanted:
            raise ValueError("%s was not asked for" % name)
    made = []
    with _launch_stream_context(x, stream):
        for name, t, like, wanted in (("dx", dx, x, input_grad), ("dw_gate", dw_gate, w_gate, weight_grads),
                                      ("dw_up", dw_up, w_up, weight_grads)):
            if t is not None:
                _ff_like(t, like.shape, like.dtype, name)
            elif wanted:
                t = like.new_empty(like.shape)
            made.append(t)
        ws_bytes = 0
        if workspace is None:
            ws_bytes = int(lib.dit_gated_feed_forward_backward_workspace_size(args))
            if ws_bytes < 0:
                raise QkrError(ws_bytes, strerror(ws_bytes))
            if ws_bytes > 0:
                workspace = x.new_empty(ws_bytes, dtype=torch.uint8)
        else:
            ws_bytes = workspace.numel() * workspace.element_size()
    dx, dw_gate, dw_up = made
    ctx, stream_ptr = _call_context(x, (dh, w_gate, w_up, gate, up, dx, dw_gate, dw_up, workspace), stream)
    with ctx:
        status = lib.dit_gated_feed_forward_backward(
            args, _ptr(dh), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(gate), _ptr(up), _ptr(dx), _ptr(dw_gate),
            _ptr(dw_up), _ptr(workspace), ws_bytes, stream_ptr)
    _check(status)
    return dx, dw_gate, dw_up
