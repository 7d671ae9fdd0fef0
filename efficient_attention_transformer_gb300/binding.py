"""ctypes binding of libflashgau (see include/flash_gau.h).

Argument marshalling only: tensors are checked for device, dtype and
contiguity and their data pointers handed to the C entry points; every step
of the computation runs in the library's CUDA kernels.  Loading fails loudly
when the library has not been built.
"""

import collections
import ctypes
import os

import numpy as np
import torch

from .build import LIB as _LIB_PATH

FP32 = 0
BF16 = 1

OK = 0
EINVAL = -1
ENOTSUP = -2
EWORKSPACE = -3
ECUDA = -4
EDEVICE = -5
ETIMEOUT = -6

MEAN = 0
SUM = 1

NORM_NONE = 0
NORM_LAYER = 1
NORM_SCALE = 2

# Every function the header declares; the library must export all of them.
EXPORTED = (
    "flash_gau_workspace_layout_query",
    "flash_gau_workspace_bytes",
    "flash_gau_forward",
    "flash_gau_forward_timed",
    "flash_gau_num_stages",
    "flash_gau_stage_name",
    "flash_gau_workspace_status",
    "flash_gau_strerror",
    "flash_gau_version",
    "flash_gau_forward_noalloc",
    "flash_gau_block_forward",
    "flash_gau_rope_toeplitz_bias",
    "flash_gau_backward_workspace_bytes",
    "flash_gau_backward",
    "flash_gau_decode_state_bytes",
    "flash_gau_decode_step",
    "flash_gau_forward_segmented",
    "flash_gau_forward_host_workspace_bytes",
    "flash_gau_forward_host",
    "flash_gau_selftest_bounded_wait",
    "flash_gau_xent_workspace_bytes",
    "flash_gau_xent",
    "flash_gau_residual_norm",
    "flash_gau_residual_norm_backward_workspace_bytes",
    "flash_gau_residual_norm_backward",
    "flash_gau_adamw_step",
    "flash_gau_adamw_moments",
    "flash_gau_bucket_bias",
    "flash_gau_bucket_bias_backward",
    "flash_gau_checkpoint_pack",
    "flash_gau_checkpoint_restore",
    "flash_gau_checkpoint_backward_workspace_bytes",
    "flash_gau_checkpoint_backward",
    "flash_gau_sample",
)

# Capacity of the static scratch behind flash_gau_forward_noalloc.
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


class Segments(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("average", ctypes.c_int)]


class Weights(ctypes.Structure):
    _fields_ = [
        ("W_uvz", ctypes.c_void_p),
        ("W_o", ctypes.c_void_p),
        ("gamma", ctypes.c_void_p),
        ("beta", ctypes.c_void_p),
        ("relpos", ctypes.c_void_p),
        ("d", ctypes.c_int),
        ("e", ctypes.c_int),
        ("s", ctypes.c_int),
        ("lin_scale", ctypes.c_float),
        ("local_scale", ctypes.c_float),
    ]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("total_bytes", "status", "U", "V", "heads", "state", "prefix", "gated",
                 "bias", "xn", "rope")]


class Block(ctypes.Structure):
    """flash_gau_block: the flash_block options (norm, RoPE, residual)."""
    _fields_ = [
        ("norm", ctypes.c_int),
        ("norm_g", ctypes.c_void_p),
        ("norm_b", ctypes.c_void_p),
        ("norm_eps", ctypes.c_float),
        ("rope", ctypes.c_int),
        ("rope_base", ctypes.c_float),
        ("pos_offset", ctypes.c_int),
        ("residual", ctypes.c_int),
    ]


class Residual(ctypes.Structure):
    """flash_gau_residual: norms, scale and gate of the residual stream."""
    _fields_ = [
        ("post", ctypes.c_int),
        ("norm", ctypes.c_int),
        ("post_g", ctypes.c_void_p),
        ("post_b", ctypes.c_void_p),
        ("norm_g", ctypes.c_void_p),
        ("norm_b", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("gate", ctypes.c_void_p),
        ("eps", ctypes.c_float),
    ]


class ResidualGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("dh", "dy", "dgate", "dscale", "dpost_g", "dpost_b", "dnorm_g", "dnorm_b")]


class XentOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("total", "loss", "lse", "dX", "dW")]


class AdamWTensor(ctypes.Structure):
    _fields_ = [
        ("p", ctypes.c_void_p),
        ("copy", ctypes.c_void_p),
        ("g", ctypes.c_void_p),
        ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("m_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("n", ctypes.c_longlong),
        ("g_dtype", ctypes.c_int),
        ("weight_decay", ctypes.c_float),
    ]


_ADAMW_TENSOR = np.dtype(AdamWTensor)


class AdamWHyper(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("step", ctypes.c_longlong),
        ("state_bits", ctypes.c_int),
        ("grad_scale", ctypes.c_void_p),
    ]


class Sampling(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("temperature", "top_k", "top_p", "min_p")]


class FlashGauError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("flash_gau status %d: %s" % (status, msg))
        self.status = status


_lib = None


def lib():
    """The loaded library (loaded on first use)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                "libflashgau.so is not built (expected at %s); call "
                "efficient_attention_transformer_gb300.build.build()" % _LIB_PATH)
        L = ctypes.CDLL(_LIB_PATH)
        i, p, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        L.flash_gau_workspace_layout_query.argtypes = [i, i, i, i, i, i, i, i,
                                                       ctypes.POINTER(WorkspaceLayout)]
        L.flash_gau_workspace_layout_query.restype = i
        L.flash_gau_workspace_bytes.argtypes = [i, i, i, ctypes.POINTER(Weights), i, i]
        L.flash_gau_workspace_bytes.restype = sz
        L.flash_gau_forward.argtypes = [p, ctypes.POINTER(Weights), i, i, i, i, i, p, p, sz, p]
        L.flash_gau_forward.restype = i
        L.flash_gau_forward_timed.argtypes = [p, ctypes.POINTER(Weights), i, i, i, i, i, p, p,
                                              sz, p, ctypes.POINTER(p), i]
        L.flash_gau_forward_timed.restype = i
        L.flash_gau_num_stages.argtypes = [i, i]
        L.flash_gau_num_stages.restype = i
        L.flash_gau_stage_name.argtypes = [i, i, i]
        L.flash_gau_stage_name.restype = ctypes.c_char_p
        L.flash_gau_workspace_status.argtypes = [p, p]
        L.flash_gau_workspace_status.restype = i
        L.flash_gau_strerror.argtypes = [i]
        L.flash_gau_strerror.restype = ctypes.c_char_p
        L.flash_gau_version.argtypes = []
        L.flash_gau_version.restype = i
        L.flash_gau_forward_noalloc.argtypes = [p, ctypes.POINTER(Weights), i, i, i, i, i, p, p]
        L.flash_gau_forward_noalloc.restype = i
        L.flash_gau_block_forward.argtypes = [p, ctypes.POINTER(Weights), ctypes.POINTER(Block),
                                              i, i, i, i, i, p, p, sz, p]
        L.flash_gau_block_forward.restype = i
        L.flash_gau_forward_segmented.argtypes = [p, ctypes.POINTER(Weights),
                                                  ctypes.POINTER(Segments), i, i, i, i, i, p,
                                                  p, sz, p]
        L.flash_gau_forward_segmented.restype = i
        L.flash_gau_forward_host_workspace_bytes.argtypes = [i, i, i, ctypes.POINTER(Weights),
                                                             i, i]
        L.flash_gau_forward_host_workspace_bytes.restype = sz
        L.flash_gau_forward_host.argtypes = [p, ctypes.POINTER(Weights), i, i, i, i, i, p, p,
                                             sz, p]
        L.flash_gau_forward_host.restype = i
        L.flash_gau_selftest_bounded_wait.argtypes = [i, p, p]
        L.flash_gau_selftest_bounded_wait.restype = i
        L.flash_gau_rope_toeplitz_bias.argtypes = [p, p, i, i, ctypes.c_float, p, p]
        L.flash_gau_rope_toeplitz_bias.restype = i
        L.flash_gau_backward_workspace_bytes.argtypes = [i, i, i, ctypes.POINTER(Weights), i, i]
        L.flash_gau_backward_workspace_bytes.restype = sz
        L.flash_gau_backward.argtypes = [p, p, ctypes.POINTER(Weights), i, i, i, i, i,
                                         ctypes.POINTER(Grads), p, sz, p]
        L.flash_gau_backward.restype = i
        L.flash_gau_decode_state_bytes.argtypes = [i, i, ctypes.POINTER(Weights), i]
        L.flash_gau_decode_state_bytes.restype = sz
        L.flash_gau_decode_step.argtypes = [p, ctypes.POINTER(Weights), i, i, i, p, sz, p, p]
        L.flash_gau_decode_step.restype = i
        ll = ctypes.c_longlong
        L.flash_gau_xent_workspace_bytes.argtypes = [ll, i, i, i, i]
        L.flash_gau_xent_workspace_bytes.restype = sz
        L.flash_gau_xent.argtypes = [p, p, p, ll, i, i, i, i, ctypes.c_float,
                                     ctypes.POINTER(XentOut), p, sz, p]
        L.flash_gau_xent.restype = i
        L.flash_gau_residual_norm.argtypes = [p, p, ctypes.POINTER(Residual), ll, i, i, p, p, p]
        L.flash_gau_residual_norm.restype = i
        L.flash_gau_residual_norm_backward_workspace_bytes.argtypes = [ll, i]
        L.flash_gau_residual_norm_backward_workspace_bytes.restype = sz
        L.flash_gau_residual_norm_backward.argtypes = [p, p, p, p, ctypes.POINTER(Residual), ll, i,
                                                       i, ctypes.POINTER(ResidualGrads), p, sz, p]
        L.flash_gau_residual_norm_backward.restype = i
        L.flash_gau_adamw_step.argtypes = [ctypes.POINTER(AdamWTensor), i,
                                           ctypes.POINTER(AdamWHyper), p]
        L.flash_gau_adamw_step.restype = i
        L.flash_gau_adamw_moments.argtypes = [ctypes.POINTER(AdamWTensor), i, ctypes.POINTER(p),
                                              ctypes.POINTER(p), p]
        L.flash_gau_adamw_moments.restype = i
        L.flash_gau_bucket_bias.argtypes = [p, i, i, i, i, i, p, p]
        L.flash_gau_bucket_bias.restype = i
        L.flash_gau_bucket_bias_backward.argtypes = [p, i, i, i, i, i, i, p, p]
        L.flash_gau_bucket_bias_backward.restype = i
        L.flash_gau_checkpoint_pack.argtypes = [p, p, ctypes.POINTER(Residual), ll, i, i, p, p, p,
                                                p, p]
        L.flash_gau_checkpoint_pack.restype = i
        L.flash_gau_checkpoint_restore.argtypes = [p, p, ctypes.POINTER(Residual), ll, i, i, p, p,
                                                   p]
        L.flash_gau_checkpoint_restore.restype = i
        L.flash_gau_checkpoint_backward_workspace_bytes.argtypes = [ll, i]
        L.flash_gau_checkpoint_backward_workspace_bytes.restype = sz
        L.flash_gau_checkpoint_backward.argtypes = [p, p, p, p, ctypes.POINTER(Residual), ll, i, i,
                                                    ctypes.POINTER(ResidualGrads), p, sz, p]
        L.flash_gau_checkpoint_backward.restype = i
        L.flash_gau_sample.argtypes = [p, ll, ll, i, i, p, ctypes.POINTER(Sampling), p, p, p, p]
        L.flash_gau_sample.restype = i
        _lib = L
    return _lib


def strerror(status):
    return lib().flash_gau_strerror(status).decode()


def _check(status):
    if status != OK:
        raise FlashGauError(status, strerror(status))


def dtype_code(t):
    if t == torch.float32:
        return FP32
    if t == torch.bfloat16:
        return BF16
    raise TypeError("io dtype must be float32 or bfloat16, got %s" % (t,))


def workspace_layout(B, T, C, d, e, s, causal, dtype):
    """Byte offsets of the intermediates, as a dict."""
    L = WorkspaceLayout()
    _check(lib().flash_gau_workspace_layout_query(B, T, C, d, e, s, int(bool(causal)),
                                                  dtype, ctypes.byref(L)))
    return {n: getattr(L, n) for n, _ in WorkspaceLayout._fields_}


def num_stages(dtype, causal):
    return lib().flash_gau_num_stages(dtype, int(bool(causal)))


def stage_names(dtype, causal):
    return [lib().flash_gau_stage_name(dtype, int(bool(causal)), k).decode()
            for k in range(num_stages(dtype, causal))]


def _dev_ptr(t, name, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


class Grads(ctypes.Structure):
    _fields_ = [("dX", ctypes.c_void_p), ("dW_uvz", ctypes.c_void_p), ("dW_o", ctypes.c_void_p),
                ("dgamma", ctypes.c_void_p), ("dbeta", ctypes.c_void_p),
                ("drelpos", ctypes.c_void_p)]


class GauWeights:
    """Device-resident layer parameters in the layout the library expects."""

    def __init__(self, W_uvz, W_o, gamma, beta, relpos, d, e, s, lin_scale=1.0,
                 local_scale=1.0):
        self.W_uvz, self.W_o = W_uvz, W_o
        self.gamma, self.beta, self.relpos = gamma, beta, relpos
        self.d, self.e, self.s = int(d), int(e), int(s)
        self.lin_scale, self.local_scale = float(lin_scale), float(local_scale)
        self.dtype = dtype_code(W_uvz.dtype)
        f32 = torch.float32
        self.c = Weights(_dev_ptr(W_uvz, "W_uvz", W_uvz.dtype), _dev_ptr(W_o, "W_o", W_uvz.dtype),
                         _dev_ptr(gamma, "gamma", f32), _dev_ptr(beta, "beta", f32),
                         _dev_ptr(relpos, "relpos", f32), self.d, self.e, self.s,
                         self.lin_scale, self.local_scale)
        if tuple(W_uvz.shape) != (d, 2 * e + s) or tuple(W_o.shape) != (e, d):
            raise ValueError("weight shapes do not match d, e, s")
        if tuple(gamma.shape) != (4, s) or tuple(beta.shape) != (4, s):
            raise ValueError("gamma and beta must be [4, s]")

    def workspace_bytes(self, B, T, C, causal):
        n = lib().flash_gau_workspace_bytes(B, T, C, ctypes.byref(self.c), int(bool(causal)),
                                            self.dtype)
        if n == 0:
            raise FlashGauError(EINVAL, "invalid or unsupported problem")
        return n

    def new_workspace(self, B, T, C, causal, device=None):
        n = self.workspace_bytes(B, T, C, causal)
        return torch.zeros(n, dtype=torch.uint8, device=device or self.W_uvz.device)


def forward(X, weights, C, causal, out=None, workspace=None, stream=None,
            stage_events=None):
    """O = FLASH-GAU(X) through flash_gau_forward (or _timed when
    stage_events, a list of torch.cuda.Event, is given).  X: [B, T, d]."""
    if X.dim() != 3:
        raise ValueError("X must be [B, T, d]")
    B, T, d = X.shape
    if d != weights.d:
        raise ValueError("X width does not match the weights")
    if X.dtype != weights.W_uvz.dtype:
        raise ValueError("X and weights must share the io dtype")
    if weights.relpos.numel() != 2 * C - 1:
        raise ValueError("relpos must hold 2C-1 values")
    if out is None:
        out = torch.empty_like(X)
    if workspace is None:
        workspace = weights.new_workspace(B, T, C, causal, X.device)
    if stream is None:
        stream = torch.cuda.current_stream(X.device)
    sp = stream.cuda_stream
    args = (_dev_ptr(X, "X", X.dtype), ctypes.byref(weights.c), B, T, C, int(bool(causal)),
            weights.dtype, _dev_ptr(out, "out", X.dtype), _dev_ptr(workspace, "workspace"),
            workspace.numel() * workspace.element_size(), sp)
    if stage_events:
        for ev in stage_events:  # torch creates the CUDA event on first record
            if not ev.cuda_event:
                ev.record(stream)
        arr = (ctypes.c_void_p * len(stage_events))(*[ev.cuda_event for ev in stage_events])
        st = lib().flash_gau_forward_timed(*args, arr, len(stage_events))
    else:
        st = lib().flash_gau_forward(*args)
    _check(st)
    return out


def forward_segmented(X, weights, C, causal, segment_ids=None, average=False, out=None,
                      workspace=None, stream=None):
    """O = FLASH-GAU(X) with a chunk mask on the global term, through
    flash_gau_forward_segmented.  segment_ids: int32 CUDA tensor [B, T / C]
    (one id per chunk; a change of id starts a segment) or None; average:
    the mean of the visible chunk states instead of their sum."""
    if X.dim() != 3:
        raise ValueError("X must be [B, T, d]")
    B, T, d = X.shape
    if d != weights.d or X.dtype != weights.W_uvz.dtype:
        raise ValueError("X does not match the weights")
    ids = None
    if segment_ids is not None:
        if T % C != 0 or tuple(segment_ids.shape) != (B, T // C):
            raise ValueError("segment_ids must be [B, T / C]")
        ids = _dev_ptr(segment_ids, "segment_ids", torch.int32)
    seg = Segments(ids, int(bool(average)))
    if out is None:
        out = torch.empty_like(X)
    if workspace is None:
        workspace = weights.new_workspace(B, T, C, causal, X.device)
    if stream is None:
        stream = torch.cuda.current_stream(X.device)
    _check(lib().flash_gau_forward_segmented(
        _dev_ptr(X, "X", X.dtype), ctypes.byref(weights.c), ctypes.byref(seg), B, T, C,
        int(bool(causal)), weights.dtype, _dev_ptr(out, "out", X.dtype),
        _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        stream.cuda_stream))
    return out


def forward_host(X, weights, C, causal, out=None, workspace=None, stream=None):
    """O = FLASH-GAU(X) on host tensors through flash_gau_forward_host: X is
    a CPU tensor [B, T, d] (pinned for overlapped copies), the result goes to
    `out` (a CPU tensor like X; allocated pinned when None).  The call
    returns once the work is queued on `stream`; synchronise it before
    reading `out`."""
    if X.dim() != 3 or X.is_cuda:
        raise ValueError("X must be a CPU tensor [B, T, d]")
    if not X.is_contiguous():
        raise ValueError("X must be contiguous")
    B, T, d = X.shape
    if d != weights.d or X.dtype != weights.W_uvz.dtype:
        raise ValueError("X does not match the weights")
    if out is None:
        out = torch.empty_like(X).pin_memory()
    if out.is_cuda or out.shape != X.shape or out.dtype != X.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous CPU tensor like X")
    dev = weights.W_uvz.device
    if workspace is None:
        n = lib().flash_gau_forward_host_workspace_bytes(B, T, C, ctypes.byref(weights.c),
                                                         int(bool(causal)), weights.dtype)
        if n == 0:
            raise FlashGauError(EINVAL, "invalid or unsupported problem")
        workspace = torch.zeros(n, dtype=torch.uint8, device=dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    _check(lib().flash_gau_forward_host(
        X.data_ptr(), ctypes.byref(weights.c), B, T, C, int(bool(causal)), weights.dtype,
        out.data_ptr(), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), stream.cuda_stream))
    return out


def forward_noalloc(X, weights, C, causal, out=None, stream=None):
    """O = FLASH-GAU(X) through flash_gau_forward_noalloc: no workspace, the
    intermediates live in the library's static 32 MiB device scratch (shared
    by every call on the device; calls must not overlap on the GPU)."""
    if X.dim() != 3:
        raise ValueError("X must be [B, T, d]")
    B, T, d = X.shape
    if d != weights.d or X.dtype != weights.W_uvz.dtype:
        raise ValueError("X does not match the weights")
    if out is None:
        out = torch.empty_like(X)
    # the library picks the scratch of the current device: make it X's
    with torch.cuda.device(X.device):
        if stream is None:
            stream = torch.cuda.current_stream(X.device)
        _check(lib().flash_gau_forward_noalloc(
            _dev_ptr(X, "X", X.dtype), ctypes.byref(weights.c), B, T, C, int(bool(causal)),
            weights.dtype, _dev_ptr(out, "out", X.dtype), stream.cuda_stream))
    return out


def block_forward(X, weights, C, causal, norm=NORM_LAYER, norm_g=None, norm_b=None,
                  norm_eps=1e-5, rope=True, rope_base=10000.0, pos_offset=0, residual=True,
                  out=None, workspace=None, stream=None):
    """Y = X + layer(norm(X)) with RoPE on the heads, through
    flash_gau_block_forward.  norm_g / norm_b: fp32 CUDA tensors ([d] for
    LayerNorm, [1] for ScaleNorm's g; norm_b may be None)."""
    if X.dim() != 3:
        raise ValueError("X must be [B, T, d]")
    B, T, d = X.shape
    if d != weights.d or X.dtype != weights.W_uvz.dtype:
        raise ValueError("X does not match the weights")
    f32 = torch.float32
    blk = Block(int(norm),
                _dev_ptr(norm_g, "norm_g", f32) if norm_g is not None else None,
                _dev_ptr(norm_b, "norm_b", f32) if norm_b is not None else None,
                float(norm_eps), int(bool(rope)), float(rope_base), int(pos_offset),
                int(bool(residual)))
    if out is None:
        out = torch.empty_like(X)
    if workspace is None:
        workspace = weights.new_workspace(B, T, C, causal, X.device)
    if stream is None:
        stream = torch.cuda.current_stream(X.device)
    _check(lib().flash_gau_block_forward(
        _dev_ptr(X, "X", X.dtype), ctypes.byref(weights.c), ctypes.byref(blk), B, T, C,
        int(bool(causal)), weights.dtype, _dev_ptr(out, "out", X.dtype),
        _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        stream.cuda_stream))
    return out


def workspace_status(workspace, stream=None):
    """Synchronises and returns (and clears) the kernels' status word."""
    if stream is None:
        stream = torch.cuda.current_stream(workspace.device)
    return lib().flash_gau_workspace_status(_dev_ptr(workspace, "workspace"), stream.cuda_stream)


def rope_toeplitz_bias(a, b, C, rope_base=10000.0, out=None, stream=None):
    """The layer's relative-position table [2C-1] (fp32, device) of the RoPE
    bias construction from the learned vectors a, b ([m] fp32 CUDA tensors),
    through flash_gau_rope_toeplitz_bias."""
    f32 = torch.float32
    if a.shape != b.shape or a.dim() != 1:
        raise ValueError("a and b must be vectors of the same length")
    if out is None:
        out = torch.empty(2 * C - 1, dtype=f32, device=a.device)
    if stream is None:
        stream = torch.cuda.current_stream(a.device)
    _check(lib().flash_gau_rope_toeplitz_bias(
        _dev_ptr(a, "a", f32), _dev_ptr(b, "b", f32), a.numel(), C, float(rope_base),
        _dev_ptr(out, "out", f32), stream.cuda_stream))
    return out


def backward(X, dO, weights, C, causal, workspace=None, stream=None):
    """Gradients of sum(dO * O) through flash_gau_backward: a dict with dX
    (io type) and dW_uvz, dW_o, dgamma, dbeta, drelpos (fp32), on X's
    device."""
    if X.dim() != 3 or dO.shape != X.shape:
        raise ValueError("X and dO must be [B, T, d]")
    B, T, d = X.shape
    if d != weights.d or X.dtype != weights.W_uvz.dtype or dO.dtype != X.dtype:
        raise ValueError("X, dO and the weights must agree")
    f32, dev = torch.float32, X.device
    e, s = weights.e, weights.s
    out = dict(dX=torch.empty_like(X),
               dW_uvz=torch.empty(d, 2 * e + s, dtype=f32, device=dev),
               dW_o=torch.empty(e, d, dtype=f32, device=dev),
               dgamma=torch.empty(4, s, dtype=f32, device=dev),
               dbeta=torch.empty(4, s, dtype=f32, device=dev),
               drelpos=torch.empty(2 * C - 1, dtype=f32, device=dev))
    g = Grads(*(_dev_ptr(out[k], k) for k in ("dX", "dW_uvz", "dW_o", "dgamma", "dbeta",
                                             "drelpos")))
    n = lib().flash_gau_backward_workspace_bytes(B, T, C, ctypes.byref(weights.c),
                                                 int(bool(causal)), weights.dtype)
    if n == 0:
        raise FlashGauError(EINVAL, "invalid or unsupported problem")
    if workspace is None:
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    _check(lib().flash_gau_backward(
        _dev_ptr(X, "X", X.dtype), _dev_ptr(dO, "dO", X.dtype), ctypes.byref(weights.c), B, T, C,
        int(bool(causal)), weights.dtype, ctypes.byref(g), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), stream.cuda_stream))
    return out


class Decoder:
    """B sequences decoded one token per call through flash_gau_decode_step;
    the state lives on the weights' device and starts all sequences at
    position 0."""

    def __init__(self, weights, B, C):
        self.weights, self.B, self.C = weights, int(B), int(C)
        n = lib().flash_gau_decode_state_bytes(self.B, self.C, ctypes.byref(weights.c),
                                               weights.dtype)
        if n == 0:
            raise FlashGauError(EINVAL, "invalid or unsupported decode problem")
        self.state = torch.zeros(n, dtype=torch.uint8, device=weights.W_uvz.device)

    def reset(self):
        self.state.zero_()

    def step(self, x, out=None, stream=None):
        """x: [B, d] in the io type; returns the [B, d] outputs."""
        if tuple(x.shape) != (self.B, self.weights.d) or x.dtype != self.weights.W_uvz.dtype:
            raise ValueError("x must be [B, d] in the weights' type")
        if out is None:
            out = torch.empty_like(x)
        if stream is None:
            stream = torch.cuda.current_stream(x.device)
        _check(lib().flash_gau_decode_step(
            _dev_ptr(x, "x", x.dtype), ctypes.byref(self.weights.c), self.B, self.C,
            self.weights.dtype, _dev_ptr(self.state, "state"), self.state.numel(),
            _dev_ptr(out, "out", x.dtype), stream.cuda_stream))
        return out


def _elsewhere(device, stream):
    """Whether a call on `device` needs _scope: a stream of its own, or another
    device than the current one."""
    return stream is not None or device.index != torch._C._cuda_getDevice()


def _scope(device, stream):
    """Context of one call on `device`: the device is current, and where a
    stream is given it is too, so that what the call allocates belongs to it."""
    if stream is not None and stream.device != device:
        raise ValueError("the stream must be one of %s" % device)
    return torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device)


def _stream(device):
    """The current stream of the device, as the library takes it."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _like(t, name, shape, dtype, index):
    """Pointer of a tensor of this shape and type on device `index`, or None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.get_device() != index:
        raise ValueError("%s must be %s %s on device %d" % (name, tuple(shape), dtype, index))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _param(t, name, n, index):
    """Pointer of n fp32 values on device `index`."""
    if t.numel() != n or t.get_device() != index or t.dtype != torch.float32:
        raise ValueError("%s must hold %d fp32 values on device %d" % (name, n, index))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _residual(shape, dtype, index, post_norm, post_g, post_b, gate, scale, norm, norm_g, norm_b,
              eps):
    d = shape[-1]
    if post_g is not None:
        post_g = _param(post_g, "post_g", d if post_norm == NORM_LAYER else 1, index)
    if post_b is not None:
        post_b = _param(post_b, "post_b", d, index)
    if norm_g is not None:
        norm_g = _param(norm_g, "norm_g", d if norm == NORM_LAYER else 1, index)
    if norm_b is not None:
        norm_b = _param(norm_b, "norm_b", d, index)
    if scale is not None:
        scale = _param(scale, "scale", d, index)
    return Residual(post_norm, norm, post_g, post_b, norm_g, norm_b, scale,
                    _like(gate, "gate", shape, dtype, index), eps)


def residual_norm(h, y=None, post_norm=NORM_NONE, post_g=None, post_b=None, gate=None, scale=None,
                  norm=NORM_LAYER, norm_g=None, norm_b=None, eps=1e-5, out_r=None, out_n=None,
                  stream=None):
    """(r, n) with r = h + scale * gate * post(y) and n = norm(r), through
    flash_gau_residual_norm.  h, y, gate: [..., d] in one io type; scale and
    the norms' parameters fp32 ([d], a ScaleNorm's g [1]).  Without y only the
    norm is taken and r is h; with norm NORM_NONE n is None."""
    dtype, shape, dev = h.dtype, h.shape, h.device
    dt, hp, at = dtype_code(dtype), _dev_ptr(h, "h"), dev.index
    if _elsewhere(dev, stream):
        with _scope(dev, stream):
            return residual_norm(h, y, post_norm, post_g, post_b, gate, scale, norm, norm_g,
                                 norm_b, eps, out_r, out_n)
    o = _residual(shape, dtype, at, post_norm, post_g, post_b, gate, scale, norm, norm_g, norm_b,
                  eps)
    yp = rp = np_ = None
    if y is not None:
        yp = _like(y, "y", shape, dtype, at)
        if out_r is None:
            out_r = torch.empty_like(h)
            rp = out_r.data_ptr()
    if out_r is not None and rp is None:
        rp = _like(out_r, "out_r", shape, dtype, at)
    if out_n is not None:
        np_ = _like(out_n, "out_n", shape, dtype, at)
    elif norm != NORM_NONE:
        out_n = torch.empty_like(h)
        np_ = out_n.data_ptr()
    d = shape[-1]
    _check(lib().flash_gau_residual_norm(hp, yp, o, h.numel() // (d or 1), d, dt, rp, np_,
                                         torch._C._cuda_getCurrentRawStream(at)))
    return (h if out_r is None else out_r), out_n


_GRADS = ("dh", "dy", "dgate", "dscale", "dpost_g", "dpost_b", "dnorm_g", "dnorm_b")


def residual_norm_backward(dr, dn, r, y, post_norm=NORM_NONE, post_g=None, post_b=None, gate=None,
                           scale=None, norm=NORM_LAYER, norm_g=None, norm_b=None, eps=1e-5,
                           out=None, workspace=None, stream=None):
    """Gradients of sum(dr * r) + sum(dn * n) through
    flash_gau_residual_norm_backward: a dict with dh, dy, dgate (io type) and
    dscale, dpost_g, dpost_b, dnorm_g, dnorm_b (fp32), None for what the
    options leave out.  dr may be None (nothing else reads the stream); y is
    the forward's y, None when the forward had none.  `out`: tensors to write
    to, by the same names (dh may be dr itself, for instance)."""
    like = dr if dr is not None else dn
    if like is None:
        raise ValueError("one of dr and dn must be given")
    _dev_ptr(like, "dr" if dr is not None else "dn")
    shape, dtype, dev = like.shape, like.dtype, like.device
    dt, at, d = dtype_code(dtype), dev.index, shape[-1]
    if _elsewhere(dev, stream):
        with _scope(dev, stream):
            return residual_norm_backward(dr, dn, r, y, post_norm, post_g, post_b, gate, scale,
                                          norm, norm_g, norm_b, eps, out, workspace)
    o = _residual(shape, dtype, at, post_norm, post_g, post_b, gate, scale, norm, norm_g, norm_b,
                  eps)
    M = like.numel() // (d or 1)
    ins = [None if t is None else _like(t, name, shape, dtype, at)
           for name, t in (("dr", dr), ("dn", dn), ("r", r), ("y", y))]
    nw = lib().flash_gau_residual_norm_backward_workspace_bytes(M, d)
    if nw == 0:
        raise FlashGauError(ENOTSUP if M > 0 and d > 0 else EINVAL, "invalid or unsupported problem")
    given, out, ptrs = out or {}, {}, []
    if not given.keys() <= set(_GRADS):
        raise ValueError("out holds %s only" % ", ".join(_GRADS))
    # each is like a tensor of the forward, which is None where it has no gradient
    post_layer, norm_layer = post_norm == NORM_LAYER, norm == NORM_LAYER
    for name, src in zip(_GRADS, (like, y, gate, scale, post_g if post_norm else None,
                                  post_g if post_layer else None, norm_g if norm else None,
                                  norm_g if norm_layer else None)):
        t = given.get(name) if given else None
        if src is None:
            if t is not None:
                raise ValueError("%s is the gradient of nothing here" % name)
            p = None
        elif t is None:
            t = torch.empty_like(src)
            p = t.data_ptr()
        else:
            p = _like(t, name, src.shape, src.dtype, at)
        ptrs.append(p)
        out[name] = t
    if workspace is None:
        workspace = torch.empty(nw, dtype=torch.uint8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp, nw = _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()
    _check(lib().flash_gau_residual_norm_backward(*ins, o, M, d, dt, ResidualGrads(*ptrs), wp, nw,
                                                  torch._C._cuda_getCurrentRawStream(at)))
    return out


def xent_workspace_bytes(N, d, V, dtype, grad=True):
    """Workspace bytes of xent for N tokens and V words (dtype FP32 or BF16)."""
    n = lib().flash_gau_xent_workspace_bytes(N, d, V, dtype, int(bool(grad)))
    if n == 0:
        raise FlashGauError(EINVAL, "invalid or unsupported problem")
    return n


_XENT_OUT = ("total", "loss", "lse", "dX", "dW")


def xent(X, W, labels, reduction=MEAN, scale=1.0, grad=True, out=None, workspace=None,
         stream=None):
    """Cross entropy of softmax(X W^T) at the labels, through flash_gau_xent:
    a dict with total (a scalar), loss and lse (like labels, fp32), and with grad
    dX and dW, the gradients of total in the io type.  X: [..., d], W: [V, d],
    labels: int32, X's leading shape; a label outside [0, V) leaves its token
    out.  total is scale times the MEAN over the labelled tokens or the SUM.
    `out`: tensors to write to, by the same names (dX and dW are not looked
    at without grad).  workspace: of xent_workspace_bytes; workspace_status
    reads from it whether a kernel's wait timed out, which nothing shows where
    the call makes its own."""
    io, dev = X.dtype, X.device
    dt, xp, at = dtype_code(io), _dev_ptr(X, "X"), dev.index
    lead = labels.shape
    if W.dim() != 2 or X.shape != lead + W.shape[1:]:
        raise ValueError("X must be [..., d], W [V, d] and labels X's leading shape")
    V, d = W.shape
    wp = _like(W, "W", (V, d), io, at)
    lp = _like(labels, "labels", lead, torch.int32, at)
    if _elsewhere(dev, stream):
        with _scope(dev, stream):
            return xent(X, W, labels, reduction, scale, grad, out, workspace)
    f32 = torch.float32
    out, ptrs = dict(out) if out else {}, []
    if not out.keys() <= set(_XENT_OUT):
        raise ValueError("out holds %s only" % ", ".join(_XENT_OUT))
    for name, like, dtype in (("total", None, f32), ("loss", labels, f32), ("lse", labels, f32),
                              ("dX", X, io), ("dW", W, io))[:5 if grad else 3]:
        t = out.get(name)
        if t is not None:
            ptrs.append(_like(t, name, () if like is None else like.shape, dtype, at))
            continue
        t = out[name] = (torch.empty((), dtype=f32, device=dev) if like is None else
                         torch.empty_like(like, dtype=dtype))
        ptrs.append(t.data_ptr())
    if not grad:
        out["dX"] = out["dW"] = None
    N = labels.numel()
    if workspace is None:
        nw = xent_workspace_bytes(N, d, V, dt, grad)
        workspace = torch.empty(nw, dtype=torch.uint8, device=dev)
        ws = workspace.data_ptr()
    else:
        ws, nw = _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()
    _check(lib().flash_gau_xent(xp, wp, lp, N, d, V, dt, reduction, scale, XentOut(*ptrs), ws, nw,
                                _stream(dev)))
    return out


class AdamW:
    """AdamW over a list of fp32 parameter tensors, one launch per step
    through flash_gau_adamw_step.

    params: contiguous fp32 CUDA tensors of one device, updated in place.
    copies: for each a bf16 tensor of its shape that receives the updated
    values (the weights that a bf16 layer reads), or None; None: no copies.
    weight_decay: one value, or one for each tensor.  state_bits: 32 (fp32
    moments) or 8 (codes with a scale for each 256 elements).  m, v, m_scale,
    v_scale: lists of existing moments (a checkpoint's) in place of zeros, m
    and v together, with 8 bits all four (memory for codes, all of them zero,
    may come without scales); they are updated in place.  All of them are
    held by the memory they have here, which the handle keeps: what is put
    into its lists later, or into a tensor's .data, is not taken (step refuses
    it for the parameters)."""

    def __init__(self, params, copies=None, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                 state_bits=32, m=None, v=None, m_scale=None, v_scale=None):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        self.params = list(params)
        k = len(self.params)
        self.copies = [None] * k if copies is None else list(copies)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * k
        f32 = torch.float32
        md, vd = (f32, f32) if state_bits == 32 else (torch.int8, torch.uint8)

        def made(given, dtype, count=None):
            if given is not None:
                return list(given)
            return [torch.zeros(p.shape if count is None else count(p.numel()), dtype=dtype,
                                device=p.device) for p in self.params]

        blocks = (lambda n: -(-n // 256))
        self.m, self.v = made(m, md), made(v, vd)
        eight = state_bits == 8
        if (m is None) != (v is None) or (m_scale is None) != (v_scale is None):
            raise ValueError("existing moments are m and v together, and their scales both")
        if m_scale is not None and (m is None or not eight):
            raise ValueError("scales belong to existing 8-bit moments")
        self.m_scale = made(m_scale, f32, blocks) if eight else [None] * k
        self.v_scale = made(v_scale, f32, blocks) if eight else [None] * k
        lists = (self.copies, decay, self.m, self.v, self.m_scale, self.v_scale)
        if any(len(x) != k for x in lists):
            raise ValueError("every list must have one entry for each parameter")
        self.device = self.params[0].device if k else None
        self._shapes = [p.shape for p in self.params]
        self._params_at = [p.data_ptr() for p in self.params]
        self._array = (AdamWTensor * max(k, 1))()
        columns = np.frombuffer(self._array, dtype=_ADAMW_TENSOR)
        n = [p.numel() for p in self.params]
        columns["n"][:k], columns["weight_decay"][:k] = n, decay
        kinds = [("p", self.params, f32, n), ("m", self.m, md, n), ("v", self.v, vd, n),
                 ("copy", self.copies, torch.bfloat16, n)]
        if eight:
            scales = [blocks(x) for x in n]
            kinds += [("m_scale", self.m_scale, f32, scales), ("v_scale", self.v_scale, f32, scales)]
        begin, end = [], []
        for name, tensors, dtype, sizes in kinds:
            ptrs = [self._pointer(t, name, dtype, x) for t, x in zip(tensors, sizes)]
            columns[name][:k] = ptrs
            live = [(a, x) for a, x in zip(ptrs, sizes) if a and x]
            begin += [a for a, _ in live]
            end += [a + x * dtype.itemsize for a, x in live]
        order = np.argsort(np.array(begin, dtype=np.uint64))
        begin, end = np.array(begin, dtype=np.uint64)[order], np.array(end, dtype=np.uint64)[order]
        if (end[:-1] > begin[1:]).any():
            raise ValueError("the tensors' parameters, copies and moments must not overlap")
        if eight and m is not None and m_scale is None and any(t.any() for t in self.m + self.v):
            raise ValueError("8-bit moments that are not zero need their scales")
        # the kernels go by address, so the memory stays here whatever becomes of
        # the lists and tensors
        self._held = [t.untyped_storage() for _, tensors, _, _ in kinds for t in tensors
                      if t is not None]
        # the columns that change from step to step
        self._g, self._g_dtype = columns["g"], columns["g_dtype"]
        self.hyper = AdamWHyper(0.0, float(betas[0]), float(betas[1]), float(eps), 0, state_bits,
                                None)
        self.state_bits, self.steps = state_bits, 0

    def _pointer(self, t, name, dtype, size):
        """0 where there is none (a copy)."""
        if t is None and name == "copy":
            return 0
        ptr = _dev_ptr(t, name, dtype)
        if t.numel() != size or t.device != self.device:
            raise ValueError("%s must hold %d values on %s" % (name, size, self.device))
        return ptr

    def step(self, grads, lr, step=None, grad_scale=None, stream=None):
        """One update with `grads`, a list of fp32 or bf16 tensors like the
        parameters.  step: its number from 1 (None: one more than the last
        one's).  grad_scale: a device fp32 scalar on the gradients, or None.
        A captured step replays with the lr and the number it was captured
        with, and with grad_scale's value at the time."""
        if len(grads) != len(self.params):
            raise ValueError("one gradient is needed for each parameter")
        if not grads:
            return
        if _elsewhere(self.device, stream):
            with _scope(self.device, stream):
                return self.step(grads, lr, step, grad_scale)
        h, dev = self.hyper, self.device
        at = dev.index
        if list(map(torch.Tensor.data_ptr, self.params)) != self._params_at:
            raise ValueError("the parameters' memory is not that of the optimizer's start")
        if [g.shape for g in grads] != self._shapes or any(g.get_device() != at for g in grads):
            raise ValueError("each gradient must be like its parameter")
        if not all(map(torch.Tensor.is_contiguous, grads)):
            raise ValueError("gradients must be contiguous")
        dtypes = [dtype_code(g.dtype) for g in grads]
        self._g[:], self._g_dtype[:] = list(map(torch.Tensor.data_ptr, grads)), dtypes
        h.lr, h.step = lr, self.steps + 1 if step is None else step
        h.grad_scale = None if grad_scale is None else _param(grad_scale, "grad_scale", 1, at)
        _check(lib().flash_gau_adamw_step(self._array, len(grads), h, _stream(dev)))
        self.steps = h.step

    def moments(self, out_m=None, out_v=None, stream=None):
        """The moments' values (m, v), two lists of fp32 tensors like the
        parameters: the tensors themselves with 32-bit moments (unless out
        lists are given), decoded through flash_gau_adamw_moments with 8-bit
        ones."""
        if not self.params:
            return [], []
        if _elsewhere(self.device, stream):
            with _scope(self.device, stream):
                return self.moments(out_m, out_v)
        k, dev, ptrs = len(self.params), self.device, []
        for name, out in (("out_m", out_m), ("out_v", out_v)):
            if out is not None and len(out) != k:
                raise ValueError("%s must hold a tensor like each parameter" % name)
        if self.state_bits == 32:
            for name, out in (("out_m", out_m), ("out_v", out_v)):
                for o, p in zip(out or [], self._shapes):
                    _like(o, name, p, torch.float32, dev.index)
            for src, out in ((self.m, out_m), (self.v, out_v)):
                for a, b in zip(src, out or []):
                    b.copy_(a.view(b.shape))
            return out_m or self.m, out_v or self.v
        out_m = out_m or [torch.empty_like(p) for p in self.params]
        out_v = out_v or [torch.empty_like(p) for p in self.params]
        for name, out in (("out_m", out_m), ("out_v", out_v)):
            ptrs.append((ctypes.c_void_p * k)(*[_like(o, name, p, torch.float32, dev.index)
                                                for o, p in zip(out, self._shapes)]))
        _check(lib().flash_gau_adamw_moments(self._array, k, *ptrs, _stream(dev)))
        return out_m, out_v


def _ints(*values):
    """Refuses whole numbers that the C ABI's int does not hold, which ctypes
    would pass on without their upper bits."""
    for v in values:
        if not -0x80000000 <= v <= 0x7fffffff:
            _check(EINVAL)


def bucket_bias(table, C, causal, max_distance=128, out=None, stream=None):
    """The layer's relative position tables [..., 2C-1] from learned values
    [..., buckets] by buckets of distance (both fp32), through
    flash_gau_bucket_bias.  Each row is one layer's GauWeights.relpos."""
    dev, f32, lead = table.device, torch.float32, table.shape
    tp, at = _dev_ptr(table, "table", f32), dev.index
    if not lead:
        raise ValueError("table must be [..., buckets]")
    if _elsewhere(dev, stream):
        with _scope(dev, stream):
            return bucket_bias(table, C, causal, max_distance, out)
    buckets = lead[-1]
    H = table.numel() // (buckets or 1)
    _ints(H, buckets, max_distance, C)
    shape = lead[:-1] + (max(2 * C - 1, 0),)
    if out is None:
        out = torch.empty(shape, dtype=f32, device=dev)
        op = out.data_ptr()
    else:
        op = _like(out, "out", shape, f32, at)
    _check(lib().flash_gau_bucket_bias(tp, H, buckets, max_distance, C, 1 if causal else 0, op,
                                       torch._C._cuda_getCurrentRawStream(at)))
    return out


def bucket_bias_backward(drelpos, buckets, causal, max_distance=128, out=None, stream=None):
    """Gradient of the values by buckets through
    flash_gau_bucket_bias_backward: drelpos [2C-1] or [H, 2C-1] as bucket_bias
    gives tables, or [R, H, 2C-1], R gradients of shared tables, which are
    added up.  Returns [buckets] or [H, buckets]."""
    dev, f32, given = drelpos.device, torch.float32, drelpos.shape
    dp, at, dims = _dev_ptr(drelpos, "drelpos", f32), dev.index, len(given)
    if not 1 <= dims <= 3 or given[-1] % 2 != 1:
        raise ValueError("drelpos must be [2C-1], [H, 2C-1] or [R, H, 2C-1]")
    if _elsewhere(dev, stream):
        with _scope(dev, stream):
            return bucket_bias_backward(drelpos, buckets, causal, max_distance, out)
    R, H, C = given[0] if dims == 3 else 1, 1 if dims == 1 else given[-2], (given[-1] + 1) // 2
    _ints(R, H, buckets, max_distance, C)
    shape = (buckets,) if dims == 1 else (H, buckets)
    if out is None:
        out = torch.empty(shape, dtype=f32, device=dev)
        op = out.data_ptr()
    else:
        op = _like(out, "out", torch.Size(shape), f32, at)
    _check(lib().flash_gau_bucket_bias_backward(dp, R, H, buckets, max_distance, C,
                                                1 if causal else 0, op,
                                                torch._C._cuda_getCurrentRawStream(at)))
    return out


class Checkpoint(collections.namedtuple("Checkpoint", ("codes", "scales"))):
    """A stream kept in 8 bits: codes int8 [..., d], and scales fp32
    [..., ceil(d / 128)], one for each 128 neighbours of a row."""

    __slots__ = ()

    @staticmethod
    def empty(shape, device):
        """Room for a stream of this shape."""
        shape = tuple(shape)
        return Checkpoint(torch.empty(shape, dtype=torch.int8, device=device),
                          torch.empty(shape[:-1] + (-(-shape[-1] // 128),), dtype=torch.float32,
                                      device=device))


def _packed(packed, shape, index):
    """Pointers of a checkpoint of a stream of this shape on device `index`."""
    codes, scales = packed
    if codes is None or scales is None:
        raise ValueError("a checkpoint is its codes and their scales")
    return (_like(codes, "codes", shape, torch.int8, index),
            _like(scales, "scales", shape[:-1] + (-(-shape[-1] // 128),), torch.float32, index))


def _norm_of(norm, norm_g, norm_b, eps, d, index):
    _ints(norm, d)
    if norm_g is not None:
        norm_g = _param(norm_g, "norm_g", d if norm == NORM_LAYER else 1, index)
    if norm_b is not None:
        norm_b = _param(norm_b, "norm_b", d, index)
    return Residual(NORM_NONE, norm, None, None, norm_g, norm_b, None, None, eps)


def checkpoint_pack(h, y=None, norm=NORM_NONE, norm_g=None, norm_b=None, eps=1e-5, out=None,
                    out_r=None, out_n=None, stream=None):
    """(Checkpoint of r, r, n) with r = h + y and n = norm(r), through
    flash_gau_checkpoint_pack: residual_norm with its stream kept in 8 bits
    for the backward pass.  Without y, r is h itself; with NORM_NONE n is
    None.  out: a Checkpoint to write to."""
    dtype, shape, dev = h.dtype, h.shape, h.device
    dt, hp, at = dtype_code(dtype), _dev_ptr(h, "h"), dev.index
    if _elsewhere(dev, stream):
        with _scope(dev, stream):
            return checkpoint_pack(h, y, norm, norm_g, norm_b, eps, out, out_r, out_n)
    d = shape[-1]
    o = _norm_of(norm, norm_g, norm_b, eps, d, at)
    yp = rp = np_ = None
    if y is not None:
        yp = _like(y, "y", shape, dtype, at)
        if out_r is None:
            out_r = torch.empty_like(h)
            rp = out_r.data_ptr()
    if out_r is not None and rp is None:
        rp = _like(out_r, "out_r", shape, dtype, at)
    if out_n is not None:
        np_ = _like(out_n, "out_n", shape, dtype, at)
    elif norm != NORM_NONE:
        out_n = torch.empty_like(h)
        np_ = out_n.data_ptr()
    if out is None:
        codes = torch.empty_like(h, dtype=torch.int8)
        scales = torch.empty(shape[:-1] + (-(-d // 128),), dtype=torch.float32, device=dev)
        out, cp, sp = Checkpoint(codes, scales), codes.data_ptr(), scales.data_ptr()
    else:
        cp, sp = _packed(out, shape, at)
    _check(lib().flash_gau_checkpoint_pack(hp, yp, o, h.numel() // (d or 1), d, dt, rp, np_, cp, sp,
                                           torch._C._cuda_getCurrentRawStream(at)))
    return out, (h if out_r is None else out_r), out_n


def checkpoint_restore(packed, dtype, norm=NORM_NONE, norm_g=None, norm_b=None, eps=1e-5,
                       want_x=True, out_x=None, out_n=None, stream=None):
    """(x, n): the stream of a Checkpoint in the io type `dtype`, and n =
    norm(x) (the input of the layer's backward), through
    flash_gau_checkpoint_restore.  x is None where it is not wanted, n with
    NORM_NONE."""
    codes = packed[0]
    dt, dev, shape = dtype_code(dtype), codes.device, codes.shape
    _dev_ptr(codes, "codes", torch.int8)
    if _elsewhere(dev, stream):
        with _scope(dev, stream):
            return checkpoint_restore(packed, dtype, norm, norm_g, norm_b, eps, want_x, out_x,
                                      out_n)
    at, d, xp, np_ = dev.index, shape[-1], None, None
    o = _norm_of(norm, norm_g, norm_b, eps, d, at)
    cp, sp = _packed(packed, shape, at)
    if out_x is not None:
        xp = _like(out_x, "out_x", shape, dtype, at)
    elif want_x:
        out_x = torch.empty_like(codes, dtype=dtype)
        xp = out_x.data_ptr()
    if out_n is not None:
        np_ = _like(out_n, "out_n", shape, dtype, at)
    elif norm != NORM_NONE:
        out_n = torch.empty_like(codes, dtype=dtype)
        np_ = out_n.data_ptr()
    _check(lib().flash_gau_checkpoint_restore(cp, sp, o, codes.numel() // (d or 1), d, dt, xp, np_,
                                              torch._C._cuda_getCurrentRawStream(at)))
    return out_x, out_n


_CHECKPOINT_GRADS = ("dh", "dnorm_g", "dnorm_b")


def checkpoint_backward(dr, dn, packed, norm=NORM_LAYER, norm_g=None, norm_b=None, eps=1e-5,
                        out=None, workspace=None, stream=None):
    """Gradients of sum(dr * x) + sum(dn * norm(x)) at the stream x of a
    Checkpoint, through flash_gau_checkpoint_backward: a dict with dh (io
    type; y's gradient too), dnorm_g and dnorm_b (fp32; dnorm_b None for a
    ScaleNorm).  dr may be None.  out: tensors to write to, by the same names
    (dh may be dr or dn itself)."""
    dtype, shape, dev = dn.dtype, dn.shape, dn.device
    dt, np_, at = dtype_code(dtype), _dev_ptr(dn, "dn"), dev.index
    if _elsewhere(dev, stream):
        with _scope(dev, stream):
            return checkpoint_backward(dr, dn, packed, norm, norm_g, norm_b, eps, out, workspace)
    d, layer = shape[-1], norm == NORM_LAYER
    M = dn.numel() // (d or 1)
    o = _norm_of(norm, norm_g, norm_b, eps, d, at)
    cp, sp = _packed(packed, shape, at)
    rp = None if dr is None else _like(dr, "dr", shape, dtype, at)
    nw = lib().flash_gau_checkpoint_backward_workspace_bytes(M, d)
    if nw == 0:
        raise FlashGauError(ENOTSUP if M > 0 and d > 0 else EINVAL, "invalid or unsupported problem")
    given, out, ptrs = out or {}, {}, []
    if given:
        if not given.keys() <= set(_CHECKPOINT_GRADS):
            raise ValueError("out holds %s only" % ", ".join(_CHECKPOINT_GRADS))
        if given.get("dnorm_b") is not None and not layer:
            raise ValueError("dnorm_b is the gradient of nothing here")
    for name, src in (("dh", dn), ("dnorm_g", norm_g),
                      ("dnorm_b", (norm_g if norm_b is None else norm_b) if layer else None)):
        t = given.get(name)
        if src is None:
            p = None
        elif t is None:
            t = torch.empty_like(src)
            p = t.data_ptr()
        else:
            p = _like(t, name, src.shape, src.dtype, at)
        out[name] = t
        ptrs.append(p)
    if workspace is None:
        workspace = torch.empty(nw, dtype=torch.uint8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp, nw = _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()
    g = ResidualGrads(ptrs[0], None, None, None, None, None, ptrs[1], ptrs[2])
    _check(lib().flash_gau_checkpoint_backward(rp, np_, cp, sp, o, M, d, dt, g, wp, nw,
                                               torch._C._cuda_getCurrentRawStream(at)))
    return out


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out_token=None,
           out_logp=None, out_kept=None, stream=None):
    """(token, logp, kept) of each row of logits [..., V], through
    flash_gau_sample: the token that the row's random number u (fp32, logits'
    leading shape, in [0, 1)) draws, the logarithm of the probability with
    which it was drawn, and how many words the filters kept.  Each filter is
    a tensor like u (top_k int32, the others fp32), one value for all rows,
    or None.  Rows of a matrix may stand further apart than V."""
    dt, dev, lead, shape = dtype_code(logits.dtype), logits.device, u.shape, logits.shape
    if not shape or shape[:-1] != lead:
        raise ValueError("logits must be [..., V] and u logits' leading shape")
    V = ld = shape[-1]
    if len(shape) == 2 and logits.is_cuda and logits.stride(1) == 1 and logits.stride(0) >= V:
        lp, ld = logits.data_ptr(), logits.stride(0)
    else:
        lp = _dev_ptr(logits, "logits")
    if _elsewhere(dev, stream):
        with _scope(dev, stream):
            return sample(logits, u, temperature, top_k, top_p, min_p, out_token, out_logp,
                          out_kept)
    _ints(V)
    at, f32, i32 = dev.index, torch.float32, torch.int32
    up = _like(u, "u", lead, f32, at)
    held, ptrs = [], []  # tensors made of single values live until the launch
    for name, t, dtype in (("temperature", temperature, f32), ("top_k", top_k, i32),
                           ("top_p", top_p, f32), ("min_p", min_p, f32)):
        if t is None:
            ptrs.append(None)
            continue
        if not isinstance(t, torch.Tensor):
            t = torch.full(lead, t, dtype=dtype, device=dev)
            held.append(t)
        ptrs.append(_like(t, name, lead, dtype, at))
    settings = Sampling(*ptrs)
    if out_token is None:
        out_token = torch.empty_like(u, dtype=i32)
        tp = out_token.data_ptr()
    else:
        tp = _like(out_token, "out_token", lead, i32, at)
    if out_logp is None:
        out_logp = torch.empty_like(u)
        gp = out_logp.data_ptr()
    else:
        gp = _like(out_logp, "out_logp", lead, f32, at)
    if out_kept is None:
        out_kept = torch.empty_like(u, dtype=i32)
        kp = out_kept.data_ptr()
    else:
        kp = _like(out_kept, "out_kept", lead, i32, at)
    _check(lib().flash_gau_sample(lp, ld, u.numel(), V, dt, up, settings, tp, gp, kp,
                                  torch._C._cuda_getCurrentRawStream(at)))
    return out_token, out_logp, out_kept
