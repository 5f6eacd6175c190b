"""Python binding of libsaf.so (include/saf.h): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module only
allocates outputs and workspace with torch, passes raw device pointers and
the current CUDA stream through ctypes, and turns status codes into
exceptions.  It raises when the library is missing: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsaf.so")

SAF_OK, SAF_ERR_INVALID_ARG, SAF_ERR_UNSUPPORTED, SAF_ERR_WORKSPACE, SAF_ERR_CUDA, SAF_ERR_TIMEOUT = range(6)
HEAD_DIM = 64

# Every symbol include/saf.h declares, with its ctypes signature.
_vp, _sz, _i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
SIGNATURES = {
    "saf_status_string": ([_i], ctypes.c_char_p),
    "saf_version": ([], _i),
    "saf_workspace_size": ([_i, _i, _i, _i, _i], _sz),
    "saf_workspace_size_gqa": ([_i, _i, _i, _i, _i, _i], _sz),
    "saf_replaced_lognorm": ([_vp, _vp, _vp, _i, _i, _vp, _vp], _i),
    "saf_mixed_attn_fwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "saf_mixed_attn_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                            _vp, _vp, _vp, _i, _vp, _sz, _vp], _i),
    "saf_mixed_attn_fwd_gqa": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp],
                               _i),
    "saf_mixed_attn_bwd_gqa": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                _vp, _vp, _vp, _i, _vp, _sz, _vp], _i),
    "saf_device_status": ([_vp, _sz, _vp], _i),
    "saf_selftest_serving_wait_limit": ([ctypes.c_longlong], _i),
    "saf_selftest_wait_timeout": ([_vp, _sz, ctypes.c_longlong, _vp], _i),
    "saf_replaced_pattern_grad": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp], _i),
    "saf_calibration_workspace_size": ([_i, _i, _i], _sz),
    "saf_fit_workspace_size": ([_i, _i], _sz),
    "saf_fit_pattern": ([_vp, _i, _i, _i, ctypes.c_float, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "saf_attn_calibration": ([_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp], _i),
    "saf_mixed_attn_bwd_noalloc": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                    _vp, _vp, _vp, _i, _vp], _i),
    "saf_rope_table": ([_vp, _i, _i, ctypes.c_double, _vp], _i),
    "saf_kv_append": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _i, _vp, _vp,
                       _i, _i, _i, _i, _vp], _i),
    "saf_paged_workspace_size": ([_i, _i, _i, _i, _i], _sz),
    "saf_paged_attn": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "saf_paged_attn_prefix": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i,
                               _vp, _sz, _vp], _i),
    "saf_launch_count": ([], ctypes.c_uint64),
    "saf_profile_enable": ([_i], _i),
    "saf_profile_read": ([ctypes.POINTER(_i), ctypes.POINTER(ctypes.c_float), _i], _i),
    "saf_kernel_name": ([_i], ctypes.c_char_p),
}

_lib = None


def _annotated(fn):
    """With SAF_NVTX=1 in the environment, each call is an NVTX range named
    saf.<function> (a profiler can then select one call, e.g. ncu --nvtx
    --nvtx-include); otherwise the call is unchanged."""
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        if os.environ.get("SAF_NVTX", "") in ("", "0"):
            return fn(*args, **kwargs)
        torch.cuda.nvtx.range_push("saf." + fn.__name__)
        try:
            return fn(*args, **kwargs)
        finally:
            torch.cuda.nvtx.range_pop()
    return wrapper


class SafError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Loads libsaf.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libsaf.so not found at {p}: build it with "
                           "`python -m mixed_head_causal_b200.build` (no fallback exists)")
    lib = ctypes.CDLL(p)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().saf_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != SAF_OK:
        raise SafError(status, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _mask_buffer(mask) -> Tuple[ctypes.Array, int]:
    m = torch.as_tensor(mask).to("cpu", torch.uint8).contiguous()
    buf = (ctypes.c_uint8 * max(1, m.numel())).from_buffer_copy(m.numpy().tobytes() or b"\0")
    return buf, m.numel()


def workspace_size(B: int, H: int, T: int, d_h: int = HEAD_DIM, backward: bool = False,
                   h_kv: Optional[int] = None) -> int:
    """Workspace bytes; h_kv (default H) K/V heads shared by groups of H / h_kv query heads."""
    if h_kv is None or h_kv == H:
        n = load().saf_workspace_size(B, H, T, d_h, 1 if backward else 0)
    else:
        n = load().saf_workspace_size_gqa(B, H, h_kv, T, d_h, 1 if backward else 0)
    if n == ctypes.c_size_t(-1).value:
        raise SafError(SAF_ERR_INVALID_ARG, "saf_workspace_size")
    return int(n)


def new_workspace(B: int, H: int, T: int, device, backward: bool = False, h_kv: Optional[int] = None) -> torch.Tensor:
    """A zero-initialised uint8 workspace (its 256-byte header must start at 0)."""
    n = max(256, workspace_size(B, H, T, HEAD_DIM, backward, h_kv))
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _check_layer_tensor(name: str, t: torch.Tensor, shape, dtype=torch.bfloat16) -> None:
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


@_annotated
def replaced_lognorm(alpha: torch.Tensor, rho: torch.Tensor, mask, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """log Z [H, T] of the replaced heads (other rows left as in `out`)."""
    H, T = alpha.shape
    if out is None:
        out = torch.zeros(H, T, dtype=torch.float32, device=alpha.device)
    mbuf, mh = _mask_buffer(mask)
    if mh != H:
        raise ValueError("mask length != H")
    _check(load().saf_replaced_lognorm(_ptr(alpha), _ptr(rho), ctypes.addressof(mbuf), H, T,
                                       _ptr(out), _stream_ptr(stream)), "saf_replaced_lognorm")
    return out


@_annotated
def mixed_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                   rho: torch.Tensor, mask, logz: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Forward of one mixed-head layer.  Returns (O [B,H,T,64] bf16, lse [B,H,T] fp32).

    k, v may hold fewer heads than q (H_kv dividing H): query head h then reads
    K/V head h // (H // H_kv) (grouped-query attention)."""
    B, H, T, d = q.shape
    Hkv = k.shape[1]
    _check_layer_tensor("q", q, (B, H, T, d))
    for n, t in (("k", k), ("v", v)):
        _check_layer_tensor(n, t, (B, Hkv, T, d))
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, H, T, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(B, H, T, q.device, backward=False, h_kv=Hkv)
    mbuf, mh = _mask_buffer(mask)
    if mh != H:
        raise ValueError("mask length != H")
    wsb = workspace.numel() * workspace.element_size()
    if Hkv == H:
        st = load().saf_mixed_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(alpha), _ptr(rho),
                                       _ptr(logz), ctypes.addressof(mbuf), B, H, T, d, _ptr(workspace), wsb,
                                       _stream_ptr(stream))
    else:
        st = load().saf_mixed_attn_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(alpha),
                                           _ptr(rho), _ptr(logz), ctypes.addressof(mbuf), B, H, Hkv, T, d,
                                           _ptr(workspace), wsb, _stream_ptr(stream))
    _check(st, "saf_mixed_attn_fwd")
    return out, lse


@_annotated
def mixed_attn_bwd(q, k, v, o, dout, lse, alpha, rho, mask, logz=None, grad_dtype=torch.bfloat16,
                   dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward of one mixed-head layer.  Returns (dQ, dK, dV) in grad_dtype (bf16 or fp32).

    With shared K/V (k, v holding H_kv < H heads) dK and dV have H_kv heads, each
    the sum over the query heads of its group."""
    B, H, T, d = q.shape
    Hkv = k.shape[1]
    for n, t in (("q", q), ("o", o), ("dout", dout)):
        _check_layer_tensor(n, t, (B, H, T, d))
    for n, t in (("k", k), ("v", v)):
        _check_layer_tensor(n, t, (B, Hkv, T, d))
    if grad_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("grad_dtype must be bf16 or fp32")
    gd = 1 if grad_dtype == torch.float32 else 0
    dq = torch.empty(B, H, T, d, dtype=grad_dtype, device=q.device) if dq is None else dq
    dk = torch.empty(B, Hkv, T, d, dtype=grad_dtype, device=q.device) if dk is None else dk
    dv = torch.empty(B, Hkv, T, d, dtype=grad_dtype, device=q.device) if dv is None else dv
    if workspace is None:
        workspace = new_workspace(B, H, T, q.device, backward=True, h_kv=Hkv)
    mbuf, mh = _mask_buffer(mask)
    if mh != H:
        raise ValueError("mask length != H")
    wsb = workspace.numel() * workspace.element_size()
    if Hkv == H:
        st = load().saf_mixed_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(alpha),
                                       _ptr(rho), _ptr(logz), ctypes.addressof(mbuf), B, H, T, d,
                                       _ptr(dq), _ptr(dk), _ptr(dv), gd, _ptr(workspace), wsb, _stream_ptr(stream))
    else:
        st = load().saf_mixed_attn_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                           _ptr(alpha), _ptr(rho), _ptr(logz), ctypes.addressof(mbuf), B, H, Hkv,
                                           T, d, _ptr(dq), _ptr(dk), _ptr(dv), gd, _ptr(workspace), wsb,
                                           _stream_ptr(stream))
    _check(st, "saf_mixed_attn_bwd")
    return dq, dk, dv


@_annotated
def replaced_pattern_grad(v, dout, alpha, rho, mask, logz=None, da=None, dr=None, workspace=None, stream=None):
    """Trainable pattern: (dalpha, drho) [H, T] fp32 of the replaced heads
    (rows of ordinary heads zero) for the output gradient dout."""
    B, H, T, d = v.shape
    for n, t in (("v", v), ("dout", dout)):
        _check_layer_tensor(n, t, (B, H, T, d))
    da = torch.empty(H, T, dtype=torch.float32, device=v.device) if da is None else da
    dr = torch.empty(H, T, dtype=torch.float32, device=v.device) if dr is None else dr
    if workspace is None and logz is None:
        workspace = new_workspace(B, H, T, v.device, backward=False)
    mbuf, mh = _mask_buffer(mask)
    if mh != H:
        raise ValueError("mask length != H")
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().saf_replaced_pattern_grad(_ptr(v), _ptr(dout), _ptr(alpha), _ptr(rho), _ptr(logz),
                                            ctypes.addressof(mbuf), B, H, T, d, _ptr(da), _ptr(dr),
                                            _ptr(workspace), wsb, _stream_ptr(stream)),
           "saf_replaced_pattern_grad")
    return da, dr


@_annotated
def fit_pattern(target, steps: int = 400, lr: float = 0.1, stream=None):
    """Fits a, r of Eq. (3) to target patterns [n, T, T] (fp32, causal, unit
    row sums).  Returns (a [n, T], r [n, T], mean row KL [n])."""
    if target.dim() == 2:
        target = target[None]
    n, T, T2 = target.shape
    if T != T2 or target.dtype != torch.float32 or not target.is_cuda or not target.is_contiguous():
        raise ValueError("target: expected a contiguous CUDA fp32 [n, T, T] tensor")
    a = torch.empty(n, T, dtype=torch.float32, device=target.device)
    r = torch.empty_like(a)
    kl = torch.empty(n, dtype=torch.float32, device=target.device)
    nbytes = load().saf_fit_workspace_size(n, T)
    if nbytes == ctypes.c_size_t(-1).value:
        raise SafError(SAF_ERR_INVALID_ARG, "saf_fit_workspace_size")
    ws = torch.zeros(max(256, int(nbytes)), dtype=torch.uint8, device=target.device)
    _check(load().saf_fit_pattern(_ptr(target), n, T, steps, lr, _ptr(a), _ptr(r), _ptr(kl), _ptr(ws),
                                  ws.numel(), _stream_ptr(stream)), "saf_fit_pattern")
    return a, r, kl


@_annotated
def attn_calibration(q, k, lse, a_hat=None, svar=None, workspace=None, stream=None):
    """Calibration statistics over the N samples of q, k [N,H,T,64] (lse from
    the forward of the same inputs): (A_hat [H,T,T] fp32, s_var [H] fp32), Eq. (1)."""
    N, H, T, d = q.shape
    for n, t in (("q", q), ("k", k)):
        _check_layer_tensor(n, t, (N, H, T, d))
    a_hat = torch.empty(H, T, T, dtype=torch.float32, device=q.device) if a_hat is None else a_hat
    svar = torch.empty(H, dtype=torch.float32, device=q.device) if svar is None else svar
    if workspace is None:
        nbytes = load().saf_calibration_workspace_size(H, T, d)
        if nbytes == ctypes.c_size_t(-1).value:
            raise SafError(SAF_ERR_INVALID_ARG, "saf_calibration_workspace_size")
        workspace = torch.empty(max(16, int(nbytes)), dtype=torch.uint8, device=q.device)
    _check(load().saf_attn_calibration(_ptr(q), _ptr(k), _ptr(lse), N, H, T, d, _ptr(a_hat), _ptr(svar),
                                       _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream_ptr(stream)), "saf_attn_calibration")
    return a_hat, svar


@_annotated
def mixed_attn_bwd_noalloc(q, k, v, o, dout, lse, alpha, rho, mask, logz=None, grad_dtype=torch.bfloat16,
                           dq=None, dk=None, dv=None, stream=None):
    """Backward without a workspace (the library's own fixed scratch, see
    include/saf.h): for callers that cannot allocate device memory.  Output
    tensors are still the caller's; pass them in to allocate nothing here."""
    B, H, T, d = v.shape
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_layer_tensor(n, t, (B, H, T, d))
    gd = 1 if grad_dtype == torch.float32 else 0
    dq = torch.empty(B, H, T, d, dtype=grad_dtype, device=v.device) if dq is None else dq
    dk = torch.empty(B, H, T, d, dtype=grad_dtype, device=v.device) if dk is None else dk
    dv = torch.empty(B, H, T, d, dtype=grad_dtype, device=v.device) if dv is None else dv
    mbuf, mh = _mask_buffer(mask)
    if mh != H:
        raise ValueError("mask length != H")
    _check(load().saf_mixed_attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                             _ptr(alpha), _ptr(rho), _ptr(logz), ctypes.addressof(mbuf),
                                             B, H, T, d, _ptr(dq), _ptr(dk), _ptr(dv), gd, _stream_ptr(stream)),
           "saf_mixed_attn_bwd_noalloc")
    return dq, dk, dv


# ------------------------------------------------------------------ serving
class _PagedKVStruct(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp)] + [(f"{t}_stride_{a}", ctypes.c_int64) for t in "kv"
                                           for a in ("page", "head", "slot")] + [
        (n, ctypes.c_int32) for n in ("num_pages", "page_size", "H_kv", "d_h")]


class PagedKV:
    """A paged key/value cache: k_cache, v_cache bf16 CUDA tensors of logical
    shape [num_pages, H_kv, page_size, 64] with a contiguous last axis and any
    other strides (pages may be stored slots first, or be slices of a larger
    tensor).  Made once and passed to the serving calls."""

    def __init__(self, k_cache: torch.Tensor, v_cache: torch.Tensor):
        for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 4 or t.shape[3] != HEAD_DIM or t.stride(3) != 1:
                raise ValueError(f"{n}: expected a CUDA bf16 [num_pages, H_kv, page_size, {HEAD_DIM}] tensor with a "
                                 f"contiguous last axis, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
        if k_cache.shape != v_cache.shape or k_cache.device != v_cache.device:
            raise ValueError("k_cache and v_cache differ in shape or device")
        self.k_cache, self.v_cache = k_cache, v_cache
        self.device = k_cache.device
        self.num_pages, self.h_kv, self.page_size, _ = k_cache.shape
        # the stride of an axis of one entry is never used: any valid one will do
        strides = [HEAD_DIM if t.shape[i] <= 1 else t.stride(i) for t in (k_cache, v_cache) for i in range(3)]
        self._struct = _PagedKVStruct(k_cache.data_ptr(), v_cache.data_ptr(), *strides, self.num_pages, self.page_size,
                                      self.h_kv, HEAD_DIM)
        self._addr = ctypes.addressof(self._struct)


def head_mask(mask) -> bytes:
    """A replaced-head mask as the bytes the library reads; made once, it
    spares the serving calls the conversion."""
    if isinstance(mask, bytes):
        return mask
    return bytes(1 if x else 0 for x in (mask.tolist() if isinstance(mask, torch.Tensor) else mask))


def _refuse(name, t, dtype, shape, device):
    raise ValueError(f"{name}: expected contiguous {dtype} of shape {tuple(shape)} on {device}, "
                     f"got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _check_serving(name, t, dtype, shape, device) -> int:
    """The address of a tensor that is contiguous, of this type and shape, and on `device`.  (Written for
    few attribute reads: a decode step's kernels take microseconds, and so do these checks.)"""
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _refuse(name, t, dtype, shape, device)
    return t.data_ptr()


def _check_tables(kv, page_table, seq_lens, q_lens, B, max_len):
    """(page_table, max_pages, seq_lens, q_lens, max_len) for the library."""
    device, cols = kv.device, page_table.shape[-1]
    if max_len is not None and not 0 <= max_len <= cols * kv.page_size:
        raise ValueError(f"max_len {max_len}: the page table holds {cols * kv.page_size} positions")
    return (_check_serving("page_table", page_table, torch.int32, (B, cols), device), cols,
            _check_serving("seq_lens", seq_lens, torch.int32, (B,), device),
            None if q_lens is None else _check_serving("q_lens", q_lens, torch.int32, (B,), device),
            cols * kv.page_size if max_len is None else max_len)


class _Guards:
    """Makes a serving call's device and stream the current ones, so that what
    it allocates belongs to the stream it runs on."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:     # (its kernels would run on the other device's memory)
            raise ValueError(f"stream: a stream of {stream.device}, the tensors are on {device}")
        self._guards = [torch.cuda.device(device)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for g in self._guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)


def _on_its_device(fn):
    """A serving call under its cache's device and its stream argument (nothing to do when both are current)."""
    @functools.wraps(fn)
    def wrapper(kv, stream, *args):
        if stream is None and kv.device.index == torch.cuda.current_device():
            return fn(kv, *args)
        with _Guards(kv.device, stream):
            return fn(kv, *args)
    return wrapper


def _current_stream(device) -> int:
    # torch.cuda.current_stream(device).cuda_stream, without its 3 us of wrapping
    return torch._C._cuda_getCurrentRawStream(device.index)


@_annotated
def rope_table(max_pos: int, rot_dim: int = HEAD_DIM, base: float = 10000.0, device="cuda", stream=None) -> torch.Tensor:
    """Rotation table [max_pos, rot_dim] fp32 for kv_append: cos in the first
    half of the columns, sin in the second."""
    device = torch.empty(0, device=device).device
    with _Guards(device, stream):
        table = torch.empty(max_pos, rot_dim, dtype=torch.float32, device=device)
        _check(load().saf_rope_table(_ptr(table), max_pos, rot_dim, base, _current_stream(device)), "saf_rope_table")
    return table


_pack_strides = struct.Struct("3q").pack


def _strided(name: str, t: torch.Tensor, shape, device) -> bytes:
    """The (batch, head, token) strides of a bf16 tensor of this shape, as the library reads them."""
    st = t.stride()
    if t.dtype != torch.bfloat16 or t.shape != shape or t.device != device or st[3] != 1:
        raise ValueError(f"{name}: expected bf16 of shape {tuple(shape)} with a contiguous last axis on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} strides {st} on {t.device}")
    if (st[0] | st[1] | st[2]) & 7:     # the stride of an axis of one entry is never used, and may be odd
        st = [0 if n <= 1 else x for x, n in zip(st, shape)]
    return _pack_strides(st[0], st[1], st[2])


@_annotated
def kv_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, kv: PagedKV, page_table: torch.Tensor,
              seq_lens: torch.Tensor, mask=None, q_lens: Optional[torch.Tensor] = None,
              rope: Optional[torch.Tensor] = None, interleaved: bool = False, max_len: Optional[int] = None,
              pos_offset: int = 0, q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
              n_heads: Optional[int] = None, stream=None):
    """Appends the new tokens k, v [B, H_kv, T, 64] to the cache and rotates q
    [B, H, T, 64] (or None) and k by `rope` (a [len, rot_dim] table, or None) on
    the way.  Returns (q_out, k_out).

    The inputs may be strided (slices of one projection's output).  seq_lens
    counts the cached tokens of each sequence including these; q_lens how many
    of the T are new ones of the sequence (None: all).  mask: replaced heads
    (their queries are skipped, and the keys of a K/V head that only they
    read); without q it needs n_heads, the length of the mask.  Rows of q_out and
    k_out that have no token or are skipped are left as they were (zeros where
    this call allocates q_out).  k_out is written only if passed."""
    H = q.shape[1] if q is not None else n_heads if n_heads is not None else len(mask) if mask is not None else k.shape[1]
    return _kv_append(kv, stream, q, k, v, page_table, seq_lens, mask, q_lens, rope, interleaved, max_len, pos_offset,
                      q_out, k_out, H)


@_on_its_device
def _kv_append(kv, q, k, v, page_table, seq_lens, mask, q_lens, rope, interleaved, max_len, pos_offset, q_out, k_out, H):
    B, Hkv, T, _ = k.shape
    device = kv.device
    if not 0 <= pos_offset <= 0x7fffffff:
        raise ValueError("pos_offset out of range")
    if Hkv != kv.h_kv:
        raise ValueError(f"k has {Hkv} heads, the cache {kv.h_kv}")
    if mask is not None:
        mask = head_mask(mask)
        if len(mask) != H:
            raise ValueError("mask length != H")
    table, cols, seq, ql, max_len = _check_tables(kv, page_table, seq_lens, q_lens, B, max_len)
    shape = (B, Hkv, T, HEAD_DIM)
    ks, vs = _strided("k", k, shape, device), _strided("v", v, shape, device)
    kop = None if k_out is None else _check_serving("k_out", k_out, torch.bfloat16, shape, device)
    qp = qs = qop = None
    if q is not None:
        shape = (B, H, T, HEAD_DIM)
        qp, qs = q.data_ptr(), _strided("q", q, shape, device)
        if q_out is None:
            q_out = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        qop = _check_serving("q_out", q_out, torch.bfloat16, shape, device)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope_len, rot_dim = (0, 0) if rope is None else rope.shape
    rp = None if rope is None else _check_serving("rope", rope, torch.float32, (rope_len, rot_dim), device)
    _check(load().saf_kv_append(kv._addr, qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, qop, kop, rp, rope_len, rot_dim,
                                1 if interleaved else 0, pos_offset, mask, table, cols, seq, ql, B, H, T, max_len,
                                _current_stream(device)), "saf_kv_append")
    return q_out, k_out


def paged_workspace_size(B: int, H: int, T_q: int, h_kv: int, prefix_len: int = 0) -> int:
    """Workspace bytes of paged_attn (prefix_len 0) and paged_attn_prefix."""
    n = load().saf_paged_workspace_size(B, H, h_kv, T_q, prefix_len)
    if n == ctypes.c_size_t(-1).value:
        raise SafError(SAF_ERR_INVALID_ARG, "saf_paged_workspace_size")
    return int(n)


def new_paged_workspace(kv: PagedKV, B: int, H: int, T_q: int = 1, prefix_len: int = 0) -> torch.Tensor:
    """A zeroed workspace for the paged attention calls of up to these sizes."""
    return torch.zeros(max(256, paged_workspace_size(B, H, T_q, kv.h_kv, prefix_len)), dtype=torch.uint8, device=kv.device)


@_on_its_device
def _paged(kv, q, prefix_table, prefix_len, page_table, seq_lens, alpha, rho, mask, q_lens, max_len, out, lse, workspace):
    B, H, T, d = q.shape
    device = kv.device
    shape = (B, H, T, HEAD_DIM)
    qp = _check_serving("q", q, torch.bfloat16, shape, device)
    tables = _check_tables(kv, page_table, seq_lens, q_lens, B, max_len)
    pattern_len, ap, rp = 0, None, None
    if mask is not None:
        mask = head_mask(mask)
        if len(mask) != H:
            raise ValueError("mask length != H")
        if alpha is not None and rho is not None:
            pattern_len = alpha.shape[-1]
            ap = _check_serving("alpha", alpha, torch.float32, (H, pattern_len), device)
            rp = _check_serving("rho", rho, torch.float32, (H, pattern_len), device)
        elif any(mask):
            raise ValueError("replaced heads need alpha and rho")
    # rows without a token are not written: they read as zeros where the call allocates
    new = torch.empty if q_lens is None else torch.zeros
    if out is None:
        out = new(shape, dtype=torch.bfloat16, device=device)
    if lse is None:
        lse = new((B, H, T), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = new_paged_workspace(kv, B, H, T, prefix_len)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {device}")
    head = (kv._addr, qp, _check_serving("out", out, torch.bfloat16, shape, device),
            _check_serving("lse", lse, torch.float32, (B, H, T), device), ap, rp, pattern_len, mask)
    tail = (*tables[:4], B, H, T, tables[4], workspace.data_ptr(), workspace.nbytes, _current_stream(device))
    if prefix_table is None:
        _check(load().saf_paged_attn(*head, *tail), "saf_paged_attn")
    else:
        pages = _check_serving("prefix_table", prefix_table, torch.int32, (-(-prefix_len // kv.page_size),), device)
        _check(load().saf_paged_attn_prefix(*head, pages, prefix_len, *tail), "saf_paged_attn_prefix")
    return out, lse


@_annotated
def paged_attn(q, kv: PagedKV, page_table, seq_lens, alpha=None, rho=None, mask=None, q_lens=None,
               max_len: Optional[int] = None, out=None, lse=None, workspace=None, stream=None):
    """Attention of T new tokens per sequence, q [B, H, T, 64] (one token of a
    decode step, a few drafted ones, a prompt chunk), over the cache that
    already holds them.  Returns (O [B, H, T, 64] bf16, lse [B, H, T] fp32).

    seq_lens [B], page_table [B, max_pages] int32 and q_lens (None, or [B] int32)
    are device tensors, read by the kernels; max_len bounds the lengths.  mask,
    alpha, rho: the replaced heads and their pattern ([H, pattern_len], at least
    max_len long).  A batch that mixes long chunks and single tokens is better
    given as two calls (see include/saf.h).  Callers that run many steps pass out, lse and a workspace
    (new_paged_workspace).  No gradient is kept: a cache is not trained through
    (the layer's own backward is mixed_attn_bwd)."""
    return _paged(kv, stream, q, None, 0, page_table, seq_lens, alpha, rho, mask, q_lens, max_len, out, lse, workspace)


@_annotated
def paged_attn_prefix(q, kv: PagedKV, prefix_table, prefix_len: int, page_table, seq_lens, alpha=None, rho=None,
                      mask=None, q_lens=None, max_len: Optional[int] = None, out=None, lse=None, workspace=None,
                      stream=None):
    """paged_attn for a batch whose sequences all begin with the same
    prefix_len tokens, cached once in the pages prefix_table [ceil(prefix_len /
    page_size)] (so many entries exactly; a longer table is sliced): the other
    arguments describe what follows the prefix."""
    if not 0 <= prefix_len <= 0x7fffffff:
        raise ValueError("prefix_len out of range")
    if prefix_table is None and prefix_len:
        raise ValueError("prefix_table: a prefix needs its pages")
    return _paged(kv, stream, q, prefix_table, prefix_len, page_table, seq_lens, alpha, rho, mask, q_lens, max_len, out, lse,
                  workspace)


def device_status(workspace: torch.Tensor, stream=None) -> int:
    """Reads and clears the device error word of `workspace` (synchronous: waits
    for `stream`, by default the current stream of the workspace's device)."""
    with _Guards(workspace.device, stream):
        return int(load().saf_device_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                            _current_stream(workspace.device)))


def selftest_wait_timeout(workspace: torch.Tensor, limit_cycles: int = 1 << 20, stream=None) -> None:
    """Enqueues a bounded device wait that nothing completes (it sets the
    workspace's error word when it gives up; see device_status)."""
    _check(load().saf_selftest_wait_timeout(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                            int(limit_cycles), _stream_ptr(stream)), "saf_selftest_wait_timeout")


def selftest_serving_wait_limit(limit_cycles: int = 0) -> None:
    """Bounds the waits of paged attention calls made from now on (0: the
    default): a test's way to make one give up (see device_status)."""
    _check(load().saf_selftest_serving_wait_limit(int(limit_cycles)), "saf_selftest_serving_wait_limit")


def launch_count() -> int:
    """Kernels the library has enqueued since it was loaded."""
    return int(load().saf_launch_count())


def profile_enable(max_launches: int) -> None:
    """Start (max_launches > 0) or stop (0) per-kernel event timing."""
    _check(load().saf_profile_enable(int(max_launches)), "saf_profile_enable")


def profile_read(n: int = 1 << 16):
    """[(kernel_name, milliseconds)] of the current profiling session."""
    lib = load()
    ids = (ctypes.c_int * n)()
    ms = (ctypes.c_float * n)()
    got = lib.saf_profile_read(ids, ms, n)
    if got < 0:
        raise SafError(SAF_ERR_CUDA, "saf_profile_read")
    return [(lib.saf_kernel_name(ids[i]).decode(), float(ms[i])) for i in range(min(got, n))]
