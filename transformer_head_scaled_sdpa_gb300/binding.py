"""ctypes binding of libmha.so (C ABI in ``include/mha.h``).

Argument marshalling only: every step of the attention forward runs in the
library's CUDA kernels.  Tensors are torch tensors (device memory and streams
come from PyTorch); their shapes are [B, L, H, d_k].  If the library has not
been built, or cannot be loaded, every call raises: there is no fallback.

``stream`` is a Stream or a raw handle (0: the default stream); the current
stream when not given.  Outputs and workspaces that are not given come from the
current stream's memory, so a call that makes any of them on another stream
first makes that stream wait for the current one; inputs are the caller's to
order.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

MHA_OK = 0
STATUS_NAMES = {
    0: "MHA_OK", 1: "MHA_ERR_NULL", 2: "MHA_ERR_SHAPE", 3: "MHA_ERR_UNSUPPORTED",
    4: "MHA_ERR_MASK", 5: "MHA_ERR_SCALE", 6: "MHA_ERR_LAUNCH", 7: "MHA_ERR_TIMEOUT",
    8: "MHA_ERR_ALIAS", 9: "MHA_ERR_WORKSPACE",
}

_lock = threading.Lock()
_lib = None

_c_p = ctypes.c_void_p
_c_i = ctypes.c_int
_FWD_ARGS = [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_p,
             ctypes.c_float, _c_p]
_FWD_LSE_ARGS = _FWD_ARGS[:4] + [_c_p] + _FWD_ARGS[4:]


class MhaError(RuntimeError):
    """A non-zero mha_status from the library."""

    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: {STATUS_NAMES.get(self.code, self.code)} "
                         f"({mha_status_string(self.code)})")


def library_path() -> str:
    return _build.LIB_PATH


def lib():
    """The loaded libmha.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it first "
                    "(python -m transformer_head_scaled_sdpa_gb300.build)")
            h = ctypes.CDLL(path)
            h.mha_fwd.restype = _c_i
            h.mha_fwd.argtypes = _FWD_ARGS
            h.mha_fwd_f32.restype = _c_i
            h.mha_fwd_f32.argtypes = _FWD_ARGS
            h.mha_fwd_lse.restype = _c_i
            h.mha_fwd_lse.argtypes = _FWD_LSE_ARGS
            h.mha_fwd_f32_lse.restype = _c_i
            h.mha_fwd_f32_lse.argtypes = _FWD_LSE_ARGS
            h.mha_layer_fwd.restype = _c_i
            h.mha_layer_fwd.argtypes = [_c_p] * 5 + [_c_i] * 7 + [_c_p, ctypes.c_float, _c_p,
                                                                   ctypes.c_size_t, _c_p]
            h.mha_layer_workspace_bytes.restype = ctypes.c_size_t
            h.mha_layer_workspace_bytes.argtypes = [_c_i] * 6
            h.mha_gemm_bf16.restype = _c_i
            h.mha_gemm_bf16.argtypes = [_c_p] * 3 + [_c_i] * 3 + [ctypes.c_longlong] * 3 + [_c_p]
            for name in ("mha_fwd_dv", "mha_fwd_f32_dv"):
                getattr(h, name).restype = _c_i
                getattr(h, name).argtypes = [_c_p] * 5 + [_c_i] * 7 + [_c_p, ctypes.c_float, _c_p]
            h.mha_bwd.restype = _c_i
            h.mha_bwd.argtypes = [_c_p] * 9 + [_c_i] * 6 + [_c_p, ctypes.c_float, _c_p,
                                                            ctypes.c_size_t, _c_p]
            h.mha_bwd_workspace_bytes.restype = ctypes.c_size_t
            h.mha_bwd_workspace_bytes.argtypes = [_c_i] * 5
            h.mha_decode.restype = _c_i
            h.mha_decode.argtypes = [_c_p] * 5 + [_c_i] * 4 + [_c_p, ctypes.c_float, _c_p,
                                                               ctypes.c_size_t, _c_p]
            h.mha_decode_static.restype = _c_i
            h.mha_decode_static.argtypes = [_c_p] * 5 + [_c_i] * 4 + [_c_p, ctypes.c_float, _c_p]
            h.mha_decode_static_scratch_bytes.restype = ctypes.c_size_t
            h.mha_decode_static_scratch_bytes.argtypes = []
            h.mha_decode_workspace_bytes.restype = ctypes.c_size_t
            h.mha_decode_workspace_bytes.argtypes = [_c_i] * 4
            h.mha_cache_write_f8.restype = _c_i
            h.mha_cache_write_f8.argtypes = [_c_p] * 2 + [ctypes.c_longlong] * 2 + [_c_p] * 4 + \
                [_c_i] * 5 + [_c_p] * 3
            h.mha_cache_read_f8.restype = _c_i
            h.mha_cache_read_f8.argtypes = [_c_p] * 6 + [_c_i] * 4 + [_c_p] * 2
            h.mha_decode_f8.restype = _c_i
            h.mha_decode_f8.argtypes = [_c_p] * 7 + [_c_i] * 5 + [_c_p, ctypes.c_float, _c_p,
                                                                  ctypes.c_size_t, _c_p]
            h.mha_decode_f8_workspace_bytes.restype = ctypes.c_size_t
            h.mha_decode_f8_workspace_bytes.argtypes = [_c_i] * 5
            for name, n_ptr in (("mha_decode_tree", 5), ("mha_decode_tree_f8", 7)):
                getattr(h, name).restype = _c_i
                getattr(h, name).argtypes = [_c_p] * n_ptr + [_c_i] * 6 + [_c_p] * 3 + \
                    [ctypes.c_float, _c_p, ctypes.c_size_t, _c_p]
                getattr(h, name + "_workspace_bytes").restype = ctypes.c_size_t
                getattr(h, name + "_workspace_bytes").argtypes = [_c_i] * 6
            h.mha_fwd_host_workspace_bytes.restype = ctypes.c_size_t
            h.mha_fwd_host_workspace_bytes.argtypes = [_c_i] * 6
            h.mha_fwd_host.restype = _c_i
            h.mha_fwd_host.argtypes = _FWD_ARGS[:-1] + [_c_i, _c_p, ctypes.c_size_t, _c_p]
            h.mha_selftest_timeout.restype = _c_i
            h.mha_selftest_timeout.argtypes = [_c_p]
            h.mha_debug_withhold_p.restype = None
            h.mha_debug_withhold_p.argtypes = [_c_i]
            h.mha_sync_status.restype = _c_i
            h.mha_sync_status.argtypes = [_c_p]
            h.mha_status_string.restype = ctypes.c_char_p
            h.mha_status_string.argtypes = [_c_i]
            h.mha_last_launch_info.restype = None
            h.mha_last_launch_info.argtypes = [ctypes.POINTER(_c_i)] * 4
            _lib = h
    return _lib


def mha_status_string(code: int) -> str:
    return lib().mha_status_string(int(code)).decode()


def _stream_handle(stream, made=()) -> int:
    """The stream's raw handle (the current stream's when None).  ``made``: tensors
    allocated here for the call, handed over to a stream other than the current
    one."""
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    if made and handle != torch._C._cuda_getCurrentRawStream(made[0].get_device()):
        _hand_over(made[0].get_device(), stream, made)
    return handle


def _hand_over(index, stream, made):
    """Gives tensors of the current stream's memory to another stream (a Stream or
    a raw handle): it waits for the current stream, on which what is queued may
    still use that memory under another name, and the allocator does not hand
    the tensors out again before that stream is done."""
    if isinstance(stream, int):
        # (ExternalStream takes handle 0, the default stream, for no stream at all)
        stream = (torch.cuda.ExternalStream(stream, device=index) if stream
                  else torch.cuda.default_stream(index))
    stream.wait_stream(torch.cuda.current_stream(index))
    for t in made:
        t.record_stream(stream)


def _shape(q, k, v, allow_dv=False):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, L, H, d_k]")
    B, Lq, H, d = q.shape
    Lk = k.shape[1]
    d_v = v.shape[3] if allow_dv else d
    if tuple(k.shape) != (B, Lk, H, d) or tuple(v.shape) != (B, Lk, H, d_v):
        raise ValueError(f"k {tuple(k.shape)} / v {tuple(v.shape)} do not match q {tuple(q.shape)}")
    return B, H, Lq, Lk, d


def _check_tensor(t, name, dtype, device_kind):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != device_kind:
        raise ValueError(f"{name} must be on {device_kind}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _call_fwd(fn_name, dtype, q, k, v, out, mask_kind, key_lens, scale, stream,
              lse=None, want_lse=False):
    B, H, Lq, Lk, d = _shape(q, k, v, allow_dv=True)
    d_v = v.shape[3]
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_tensor(t, n, dtype, "cuda")
    made = []
    if out is None:
        out = torch.empty((B, Lq, H, d_v), dtype=dtype, device=q.device)
        made.append(out)
    _check_tensor(out, "out", dtype, "cuda")
    if tuple(out.shape) != (B, Lq, H, d_v):
        raise ValueError("out must be [B, Lq, H, d_v]")
    lens_ptr = None
    if key_lens is not None:
        _check_tensor(key_lens, "key_lens", torch.int32, "cuda")
        if tuple(key_lens.shape) != (B,):
            raise ValueError("key_lens must be [B]")
        lens_ptr = key_lens.data_ptr()
    if d_v != d:
        # value rows of their own width: the *_dv entry (lse optional)
        if want_lse:
            if lse is None:
                lse = torch.empty((B, H, Lq), dtype=torch.float32, device=q.device)
                made.append(lse)
            _check_tensor(lse, "lse", torch.float32, "cuda")
            if tuple(lse.shape) != (B, H, Lq):
                raise ValueError("lse must be [B, H, Lq]")
        fn_name += "_dv"
        rc = getattr(lib(), fn_name)(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                     lse.data_ptr() if want_lse else None, B, H, Lq, Lk, d, d_v,
                                     int(mask_kind), lens_ptr, float(scale),
                                     _stream_handle(stream, made))
        if rc != MHA_OK:
            raise MhaError(rc, fn_name)
        return (out, lse) if want_lse else out
    if not want_lse:
        rc = getattr(lib(), fn_name)(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                     B, H, Lq, Lk, d, int(mask_kind), lens_ptr, float(scale),
                                     _stream_handle(stream, made))
        if rc != MHA_OK:
            raise MhaError(rc, fn_name)
        return out
    if lse is None:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=q.device)
        made.append(lse)
    _check_tensor(lse, "lse", torch.float32, "cuda")
    if tuple(lse.shape) != (B, H, Lq):
        raise ValueError("lse must be [B, H, Lq]")
    fn_name += "_lse"
    rc = getattr(lib(), fn_name)(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                 lse.data_ptr(), B, H, Lq, Lk, d, int(mask_kind), lens_ptr,
                                 float(scale), _stream_handle(stream, made))
    if rc != MHA_OK:
        raise MhaError(rc, fn_name)
    return out, lse


def mha_fwd(q, k, v, out=None, mask_kind: int = 0, key_lens=None, scale: float = 0.0,
            stream=None, return_lse: bool = False, lse=None):
    """bf16 attention forward on the GPU (tcgen05 kernel); returns ``out``, or
    ``(out, lse)`` with ``return_lse`` (lse: float32 [B, H, Lq], natural log).
    v (and out) may have a width d_v of their own: q, k [.., d_k], v [.., d_v]."""
    return _call_fwd("mha_fwd", torch.bfloat16, q, k, v, out, mask_kind, key_lens, scale,
                     stream, lse, return_lse)


def mha_fwd_f32(q, k, v, out=None, mask_kind: int = 0, key_lens=None, scale: float = 0.0,
                stream=None, return_lse: bool = False, lse=None):
    """float32 attention forward on the GPU (SIMT kernel); returns ``out``, or
    ``(out, lse)`` with ``return_lse``."""
    return _call_fwd("mha_fwd_f32", torch.float32, q, k, v, out, mask_kind, key_lens, scale,
                     stream, lse, return_lse)


def mha_bwd(q, k, v, out, dout, lse, mask_kind: int = 0, key_lens=None, scale: float = 0.0,
            dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradient of mha_fwd (bf16): returns (dq, dk, dv) for dL/dout = ``dout``,
    given the forward's ``out`` and ``lse`` (from mha_fwd(..., return_lse=True))."""
    B, H, Lq, Lk, d = _shape(q, k, v)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _check_tensor(t, n, torch.bfloat16, "cuda")
    if tuple(out.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape):
        raise ValueError("out and dout must have q's shape")
    _check_tensor(lse, "lse", torch.float32, "cuda")
    if tuple(lse.shape) != (B, H, Lq):
        raise ValueError("lse must be [B, H, Lq]")
    given = (dq, dk, dv, workspace)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, ref, n in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
        _check_tensor(t, n, torch.bfloat16, "cuda")
        if tuple(t.shape) != tuple(ref.shape):
            raise ValueError(f"{n} must have the shape of its input")
    lens_ptr = None
    if key_lens is not None:
        _check_tensor(key_lens, "key_lens", torch.int32, "cuda")
        lens_ptr = key_lens.data_ptr()
    need = int(lib().mha_bwd_workspace_bytes(B, H, Lq, Lk, d))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check_tensor(workspace, "workspace", torch.uint8, "cuda")
    made = [t for t, g in zip((dq, dk, dv, workspace), given) if g is None]
    rc = lib().mha_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                       dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                       dv.data_ptr(), B, H, Lq, Lk, d, int(mask_kind), lens_ptr, float(scale),
                       workspace.data_ptr(), workspace.numel(), _stream_handle(stream, made))
    if rc != MHA_OK:
        raise MhaError(rc, "mha_bwd")
    return dq, dk, dv


def layer_workspace_bytes(B, Lq, Lk, d_model, H, d_k) -> int:
    return int(lib().mha_layer_workspace_bytes(B, Lq, Lk, d_model, H, d_k))


def mha_layer_fwd(x, w_qkv, w_o, H: int, mem=None, mask_kind: int = 0, key_lens=None,
                  scale: float = 0.0, y=None, workspace=None, stream=None):
    """One multi-head attention layer (bf16): y = Concat(heads) W^O with
    head_h = Attention(x W_h^Q, m W_h^K, m W_h^V), m = ``mem`` or x.
    x [B, Lq, d_model], mem [B, Lk, d_model] or None, w_qkv [d_model, 3 H d_k],
    w_o [H d_k, d_model]; returns y [B, Lq, d_model]."""
    if x.dim() != 3 or w_qkv.dim() != 2 or w_o.dim() != 2:
        raise ValueError("x must be [B, Lq, d_model], w_qkv and w_o matrices")
    B, Lq, d_model = x.shape
    hd3 = w_qkv.shape[1]
    if hd3 % (3 * H) != 0 or tuple(w_qkv.shape) != (d_model, hd3):
        raise ValueError("w_qkv must be [d_model, 3 H d_k]")
    d_k = hd3 // (3 * H)
    if tuple(w_o.shape) != (H * d_k, d_model):
        raise ValueError("w_o must be [H d_k, d_model]")
    Lk = Lq if mem is None else mem.shape[1]
    tensors = [(x, "x"), (w_qkv, "w_qkv"), (w_o, "w_o")]
    if mem is not None:
        if mem.dim() != 3 or mem.shape[0] != B or mem.shape[2] != d_model:
            raise ValueError("mem must be [B, Lk, d_model]")
        tensors.append((mem, "mem"))
    for t, n in tensors:
        _check_tensor(t, n, torch.bfloat16, "cuda")
    made = []
    if y is None:
        y = torch.empty_like(x)
        made.append(y)
    _check_tensor(y, "y", torch.bfloat16, "cuda")
    if tuple(y.shape) != tuple(x.shape):
        raise ValueError("y must have x's shape")
    lens_ptr = None
    if key_lens is not None:
        _check_tensor(key_lens, "key_lens", torch.int32, "cuda")
        lens_ptr = key_lens.data_ptr()
    need = layer_workspace_bytes(B, Lq, Lk, d_model, H, d_k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
        made.append(workspace)
    _check_tensor(workspace, "workspace", torch.uint8, "cuda")
    rc = lib().mha_layer_fwd(x.data_ptr(), mem.data_ptr() if mem is not None else None,
                             w_qkv.data_ptr(), w_o.data_ptr(), y.data_ptr(), B, Lq, Lk, d_model,
                             H, d_k, int(mask_kind), lens_ptr, float(scale), workspace.data_ptr(),
                             workspace.numel(), _stream_handle(stream, made))
    if rc != MHA_OK:
        raise MhaError(rc, "mha_layer_fwd")
    return y


def mha_gemm_bf16(a, b, c=None, stream=None):
    """c = a @ b on the library's tensor-core GEMM: a [M, K], b [K, N] bf16
    CUDA matrices whose rows may be strided (stride(1) == 1, stride(0) a
    multiple of 8 elements, e.g. column blocks of a wider matrix); c [M, N]
    (allocated when not given, else written in place, same row rules)."""
    for t, n in ((a, "a"), (b, "b")):
        if t.dim() != 2 or t.dtype != torch.bfloat16 or not t.is_cuda or t.stride(1) != 1:
            raise ValueError(f"{n} must be a row-major bf16 CUDA matrix")
    M, K = a.shape
    if b.shape[0] != K:
        raise ValueError(f"inner sizes differ: a {tuple(a.shape)}, b {tuple(b.shape)}")
    N = b.shape[1]
    made = []
    if c is None:
        c = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
        made.append(c)
    if c.dim() != 2 or tuple(c.shape) != (M, N) or c.dtype != torch.bfloat16 or c.stride(1) != 1:
        raise ValueError("c must be a row-major bf16 [M, N] matrix")
    rc = lib().mha_gemm_bf16(a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K,
                             max(a.stride(0), K), max(b.stride(0), N), max(c.stride(0), N),
                             _stream_handle(stream, made))
    if rc != MHA_OK:
        raise MhaError(rc, "mha_gemm_bf16")
    return c


def decode_workspace_bytes(B, H, Lk, d_k) -> int:
    return int(lib().mha_decode_workspace_bytes(B, H, Lk, d_k))


def mha_decode_static(q, k_cache, v_cache, cache_lens, out=None, scale: float = 0.0,
                      stream=None, return_lse: bool = False, lse=None):
    """mha_decode with the library's fixed device scratch instead of a
    workspace (calls on one device must not overlap in time)."""
    return mha_decode(q, k_cache, v_cache, cache_lens, out=out, scale=scale, stream=stream,
                      return_lse=return_lse, lse=lse, _static=True)


def mha_decode(q, k_cache, v_cache, cache_lens, out=None, scale: float = 0.0, workspace=None,
               stream=None, return_lse: bool = False, lse=None, _static: bool = False):
    """One decode step (bf16): q [B, H, d] (or [B, 1, H, d]) against the first
    cache_lens[b] rows of k_cache / v_cache [B, Lk, H, d].  Returns out
    [B, H, d] (q's shape), or (out, lse) with ``return_lse``.  ``workspace``
    (uint8 CUDA tensor) is allocated when not given."""
    if q.dim() == 4:
        if q.shape[1] != 1:
            raise ValueError("q must be [B, H, d] or [B, 1, H, d]")
    elif q.dim() != 3:
        raise ValueError("q must be [B, H, d] or [B, 1, H, d]")
    B, H, d = q.shape[0], q.shape[-2], q.shape[-1]
    if k_cache.dim() != 4 or tuple(k_cache.shape[::2]) != (B, H) or k_cache.shape[3] != d \
            or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError(f"caches {tuple(k_cache.shape)} / {tuple(v_cache.shape)} do not match q")
    Lk = k_cache.shape[1]
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _check_tensor(t, n, torch.bfloat16, "cuda")
    _check_tensor(cache_lens, "cache_lens", torch.int32, "cuda")
    if tuple(cache_lens.shape) != (B,):
        raise ValueError("cache_lens must be [B]")
    made = []
    if out is None:
        out = torch.empty_like(q)
        made.append(out)
    _check_tensor(out, "out", torch.bfloat16, "cuda")
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError("out must have q's shape")
    lse_ptr = None
    if return_lse:
        if lse is None:
            lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
            made.append(lse)
        _check_tensor(lse, "lse", torch.float32, "cuda")
        if tuple(lse.shape) != (B, H):
            raise ValueError("lse must be [B, H]")
        lse_ptr = lse.data_ptr()
    if _static:
        rc = lib().mha_decode_static(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                     out.data_ptr(), lse_ptr, B, H, Lk, d,
                                     cache_lens.data_ptr(), float(scale), _stream_handle(stream, made))
        if rc != MHA_OK:
            raise MhaError(rc, "mha_decode_static")
        return (out, lse) if return_lse else out
    need = decode_workspace_bytes(B, H, Lk, d)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        made.append(workspace)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _check_tensor(workspace, "workspace", torch.uint8, "cuda")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel()
    rc = lib().mha_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                          lse_ptr, B, H, Lk, d, cache_lens.data_ptr(), float(scale), ws_ptr,
                          ws_bytes, _stream_handle(stream, made))
    if rc != MHA_OK:
        raise MhaError(rc, "mha_decode")
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------------------
# the 8-bit cache, and steps of a few rows per sequence over a cache
# ---------------------------------------------------------------------------
_BF16, _F32, _I32, _I64, _U8 = (torch.bfloat16, torch.float32, torch.int32, torch.int64,
                                torch.uint8)
_F8 = torch.float8_e4m3fn


def _refuse(t, name, dtype, index):
    """Raises what is wrong with a tensor that _check found wrong."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if index < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be on cuda, got {t.device}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, others on cuda:{index}")
    raise ValueError(f"{name} must be contiguous")


def _check(index, tensors):
    """Checks (tensor, name, dtype) triples: dtype, contiguous, all on the CUDA
    device `index`.  (A small step costs as much on the host as on the GPU: one
    comparison each here, the words in _refuse.)"""
    for t, name, dtype in tensors:
        if t.dtype is not dtype or index < 0 or t.get_device() != index or not t.is_contiguous():
            _refuse(t, name, dtype, index)


def _call_on(index, stream, made, fn, args):
    """Calls an entry with device `index` current and its stream (the current one
    unless given).  ``made``: tensors allocated here for the call, handed over to
    a stream other than the current one."""
    # (the raw handle: building a Stream object costs more than the launch)
    handle = torch._C._cuda_getCurrentRawStream(index)
    if stream is not None:
        other = stream if isinstance(stream, int) else stream.cuda_stream
        if other != handle:
            handle = other
            if made:
                _hand_over(index, stream, made)
    if torch.cuda.current_device() == index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc:
        raise MhaError(rc, fn.__name__)


def _row_strides(t, name):
    """(token stride, sequence stride) in elements of rows [B, T, H, d] whose
    H * d values are contiguous."""
    B, T, H, d = t.shape
    if t.numel() == 0:
        return 0, 0
    if t.stride(3) != 1 or (H > 1 and t.stride(2) != d):
        raise ValueError(f"{name}'s rows of H * d_k values must be contiguous")
    token = t.stride(1) if T > 1 else H * d
    seq = t.stride(0) if B > 1 else T * token
    if token < H * d or seq < H * d:
        raise ValueError(f"{name}'s rows overlap (expanded?)")
    return token, seq


def _cache_shape(k_cache, v_cache, k_scale, v_scale):
    """Checks the shapes of an 8-bit cache; returns (B, Lk, H, d)."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache {tuple(shape)} and v_cache {tuple(v_cache.shape)} "
                         "must be [B, Lk, H, d_k] alike")
    scales = (shape[0], shape[2], shape[1])
    if k_scale.shape != scales or v_scale.shape != scales:
        raise ValueError(f"k_scale and v_scale must be [B, H, Lk] = {scales}")
    return shape


def _lens(t, name, B):
    if t.shape != (B,):
        raise ValueError(f"{name} must be [B]")
    return (t, name, _I32)


def mha_cache_write_f8(k, v, k_cache, v_cache, k_scale, v_scale, start, counts=None, stream=None):
    """Quantises new rows k, v [B, T, H, d] (bf16; rows of a packed projection
    are read in place) into the 8-bit cache at positions start[b] .. : codes
    k_cache, v_cache [B, Lk, H, d] (float8_e4m3fn), biased exponents k_scale,
    v_scale [B, H, Lk] (uint8).  ``counts`` [B] limits the tokens of a
    sequence; positions outside the cache are dropped."""
    B, Lk, H, d = _cache_shape(k_cache, v_cache, k_scale, v_scale)
    shape = k.shape
    if len(shape) != 4 or shape[0] != B or shape[2] != H or shape[3] != d or v.shape != shape:
        raise ValueError(f"k {tuple(shape)} and v {tuple(v.shape)} must be [B, T, H, d_k] of "
                         f"the cache {tuple(k_cache.shape)}")
    strides = _row_strides(k, "k")
    if _row_strides(v, "v") != strides:
        raise ValueError("k and v must have the same strides")
    index = k_cache.get_device()
    _check(index, ((k_cache, "k_cache", _F8), (v_cache, "v_cache", _F8), (k_scale, "k_scale", _U8),
                   (v_scale, "v_scale", _U8), _lens(start, "start", B)))
    if counts is not None:
        _check(index, (_lens(counts, "counts", B),))
    for t, name in ((k, "k"), (v, "v")):
        if t.dtype is not _BF16 or t.get_device() != index:
            _refuse(t, name, _BF16, index)
    _call_on(index, stream, (), lib().mha_cache_write_f8,
             (k.data_ptr(), v.data_ptr(), *strides, k_cache.data_ptr(), v_cache.data_ptr(),
              k_scale.data_ptr(), v_scale.data_ptr(), B, shape[1], H, Lk, d, start.data_ptr(),
              counts.data_ptr() if counts is not None else None))


def mha_cache_read_f8(k_cache, v_cache, k_scale, v_scale, lens, k=None, v=None, stream=None):
    """The first lens[b] positions of an 8-bit cache as bf16: returns (k, v)
    [B, Lk, H, d].  Positions from lens[b] on keep what ``k`` and ``v`` held
    (0 when they are allocated here)."""
    shape = _cache_shape(k_cache, v_cache, k_scale, v_scale)
    B, Lk, H, d = shape
    index = k_cache.get_device()
    _check(index, ((k_cache, "k_cache", _F8), (v_cache, "v_cache", _F8), (k_scale, "k_scale", _U8),
                   (v_scale, "v_scale", _U8), _lens(lens, "lens", B)))
    made = []
    out = []
    for t, name in ((k, "k"), (v, "v")):
        if t is None:
            t = torch.zeros(shape, dtype=_BF16, device=k_cache.device)
            made.append(t)
        else:
            if t.shape != shape:
                raise ValueError(f"{name} must have the cache's shape {tuple(shape)}")
            _check(index, ((t, name, _BF16),))
        out.append(t)
    k, v = out
    _call_on(index, stream, made, lib().mha_cache_read_f8,
             (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
              k.data_ptr(), v.data_ptr(), B, H, Lk, d, lens.data_ptr()))
    return k, v


def _rows_call(fn, ws_fn, q, cache_shape, tensors, ptrs, lens, extra, out, scale, workspace,
               stream, return_lse, lse, ws_args, lse_shape):
    """What the steps of a few rows have in common: checks, allocation, call."""
    B, Lk, H_kv, d = cache_shape
    q_shape = q.shape
    if q_shape[0] != B or q_shape[-1] != d or H_kv == 0 or q_shape[-2] % H_kv != 0:
        raise ValueError(f"cache {tuple(cache_shape)} does not match q {tuple(q_shape)}")
    index = q.get_device()
    _check(index, tensors)
    made = []
    if out is None:
        out = torch.empty_like(q)
        made.append(out)
    elif out.shape != q_shape:
        raise ValueError("out must have q's shape")
    else:
        _check(index, ((out, "out", _BF16),))
    if lse is not None:
        if lse.shape != lse_shape:
            raise ValueError(f"lse must be {lse_shape}")
        _check(index, ((lse, "lse", _F32),))
    elif return_lse:
        lse = torch.empty(lse_shape, dtype=_F32, device=q.device)
        made.append(lse)
    if workspace is None:
        need = ws_fn(*ws_args)
        if need:
            workspace = torch.empty(need, dtype=_U8, device=q.device)
            made.append(workspace)
    else:
        _check(index, ((workspace, "workspace", _U8),))
    _call_on(index, stream, made, fn,
             (q.data_ptr(), *ptrs, out.data_ptr(), lse.data_ptr() if return_lse else None,
              *ws_args, lens.data_ptr(), *extra, scale,
              *((None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel()))))
    return (out, lse) if return_lse else out


def decode_f8_workspace_bytes(B, H, H_kv, Lk, d_k) -> int:
    return int(lib().mha_decode_f8_workspace_bytes(B, H, H_kv, Lk, d_k))


def decode_tree_workspace_bytes(B, T, H, H_kv, Lk, d_k) -> int:
    return int(lib().mha_decode_tree_workspace_bytes(B, T, H, H_kv, Lk, d_k))


def decode_tree_f8_workspace_bytes(B, T, H, H_kv, Lk, d_k) -> int:
    return int(lib().mha_decode_tree_f8_workspace_bytes(B, T, H, H_kv, Lk, d_k))


def mha_decode_f8(q, k_cache, v_cache, k_scale, v_scale, cache_lens, out=None, scale: float = 0.0,
                  workspace=None, stream=None, return_lse: bool = False, lse=None):
    """One decode step over an 8-bit cache: q [B, H, d] (or [B, 1, H, d], bf16)
    against the first cache_lens[b] positions of k_cache, v_cache
    [B, Lk, H_kv, d] with scales [B, H_kv, Lk] (mha_cache_write_f8's format);
    query head h reads key head h // (H / H_kv).  Returns out (q's shape), or
    (out, lse) with ``return_lse`` (lse [B, H]).  ``workspace`` (uint8 CUDA
    tensor) is allocated when not given."""
    if q.dim() not in (3, 4) or (q.dim() == 4 and q.shape[1] != 1):
        raise ValueError("q must be [B, H, d] or [B, 1, H, d]")
    shape = _cache_shape(k_cache, v_cache, k_scale, v_scale)
    B, Lk, H_kv, d = shape
    H = q.shape[-2]
    h = lib()
    return _rows_call(
        h.mha_decode_f8, h.mha_decode_f8_workspace_bytes, q, shape,
        ((q, "q", _BF16), (k_cache, "k_cache", _F8), (v_cache, "v_cache", _F8),
         (k_scale, "k_scale", _U8), (v_scale, "v_scale", _U8), _lens(cache_lens, "cache_lens", B)),
        (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()),
        cache_lens, (), out, scale, workspace, stream, return_lse, lse, (B, H, H_kv, Lk, d), (B, H))


def _tree_mask(q, draft_lens, tree_mask):
    """Checks the shapes of a tree step's q, lengths and mask; returns the mask's
    and lengths' triples and pointers."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, d]")
    B, T = q.shape[0], q.shape[1]
    tensors, drafts, bits = (), None, None
    if draft_lens is not None:
        tensors = (_lens(draft_lens, "draft_lens", B),)
        drafts = draft_lens.data_ptr()
    if tree_mask is not None:
        words = (T + 63) // 64
        if tree_mask.shape != (B, T, words):
            raise ValueError(f"tree_mask must be [B, T, ceil(T / 64)] = {(B, T, words)}")
        tensors += ((tree_mask, "tree_mask", _I64),)
        bits = tree_mask.data_ptr()
    return tensors, (drafts, bits)


def mha_decode_tree(q, k_cache, v_cache, prefix_lens, draft_lens=None, tree_mask=None, out=None,
                    scale: float = 0.0, workspace=None, stream=None, return_lse: bool = False,
                    lse=None):
    """One step of a tree of T drafted tokens per sequence over a bf16 cache:
    q [B, T, H, d]; k_cache, v_cache [B, Lk, H_kv, d] hold the prefix
    (prefix_lens[b] positions, seen by every row) and drafted token j at
    position prefix_lens[b] + j.  ``tree_mask`` int64 [B, T, ceil(T / 64)]: row
    t sees drafted token j where bit j is set (None: a chain, j <= t).
    ``draft_lens`` [B]: drafted tokens per sequence (None: T); rows past them
    get output 0.  Returns out [B, T, H, d], or (out, lse [B, H, T])."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache {tuple(shape)} and v_cache {tuple(v_cache.shape)} "
                         "must be [B, Lk, H_kv, d] alike")
    tree, extra = _tree_mask(q, draft_lens, tree_mask)
    B, T, H, _ = q.shape
    h = lib()
    return _rows_call(
        h.mha_decode_tree, h.mha_decode_tree_workspace_bytes, q, shape,
        ((q, "q", _BF16), (k_cache, "k_cache", _BF16), (v_cache, "v_cache", _BF16),
         _lens(prefix_lens, "prefix_lens", B), *tree),
        (k_cache.data_ptr(), v_cache.data_ptr()), prefix_lens, extra, out, scale, workspace,
        stream, return_lse, lse, (B, T, H, shape[2], shape[1], shape[3]), (B, H, T))


def mha_decode_tree_f8(q, k_cache, v_cache, k_scale, v_scale, prefix_lens, draft_lens=None,
                       tree_mask=None, out=None, scale: float = 0.0, workspace=None, stream=None,
                       return_lse: bool = False, lse=None):
    """mha_decode_tree over an 8-bit cache (mha_cache_write_f8's format)."""
    shape = _cache_shape(k_cache, v_cache, k_scale, v_scale)
    tree, extra = _tree_mask(q, draft_lens, tree_mask)
    B, T, H, _ = q.shape
    h = lib()
    return _rows_call(
        h.mha_decode_tree_f8, h.mha_decode_tree_f8_workspace_bytes, q, shape,
        ((q, "q", _BF16), (k_cache, "k_cache", _F8), (v_cache, "v_cache", _F8),
         (k_scale, "k_scale", _U8), (v_scale, "v_scale", _U8),
         _lens(prefix_lens, "prefix_lens", B), *tree),
        (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()),
        prefix_lens, extra, out, scale, workspace, stream, return_lse, lse,
        (B, T, H, shape[2], shape[1], shape[3]), (B, H, T))


def host_workspace_bytes(B, H, Lq, Lk, d_k, elem_bytes) -> int:
    return int(lib().mha_fwd_host_workspace_bytes(B, H, Lq, Lk, d_k, elem_bytes))


def mha_fwd_host(q, k, v, out, workspace, mask_kind: int = 0, key_lens=None,
                 scale: float = 0.0, stream=None) -> int:
    """Attention on HOST tensors (pinned for async copies) through the C ABI's
    host-buffer entry: H2D copies, the kernel and the D2H copy of ``out`` all
    run on ``stream``; returns once ``out`` holds the result."""
    B, H, Lq, Lk, d = _shape(q, k, v)
    dtype = q.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("host tensors must be bf16 or float32")
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _check_tensor(t, n, dtype, "cpu")
    lens_ptr = None
    if key_lens is not None:
        _check_tensor(key_lens, "key_lens", torch.int32, "cpu")
        lens_ptr = key_lens.data_ptr()
    _check_tensor(workspace, "workspace", torch.uint8, "cuda")
    rc = lib().mha_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                            B, H, Lq, Lk, d, int(mask_kind), lens_ptr, float(scale),
                            2 if dtype == torch.bfloat16 else 4, workspace.data_ptr(),
                            workspace.numel(), _stream_handle(stream))
    if rc != MHA_OK:
        raise MhaError(rc, "mha_fwd_host")
    return rc


def mha_sync_status(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) the device status code."""
    return int(lib().mha_sync_status(_stream_handle(stream)))


def mha_selftest_timeout(stream=None) -> int:
    """Launch the bounded-wait self-test kernel (see include/mha.h)."""
    rc = lib().mha_selftest_timeout(_stream_handle(stream))
    if rc != MHA_OK:
        raise MhaError(rc, "mha_selftest_timeout")
    return rc


def mha_debug_withhold_p(on: bool) -> None:
    """Test hook: make later mha_fwd launches run out a pipeline wait."""
    lib().mha_debug_withhold_p(1 if on else 0)


def last_launch_info() -> dict:
    vals = [ctypes.c_int(0) for _ in range(4)]
    lib().mha_last_launch_info(*[ctypes.byref(x) for x in vals])
    return dict(zip(("kernels", "grid", "block", "smem"), (x.value for x in vals)))
