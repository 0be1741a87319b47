"""Python binding of libhyena_b200 (argument marshalling only).

Every function here passes device pointers, sizes and the current CUDA stream
to the C ABI declared in ``include/hyena.h``; all arithmetic runs in the
library's CUDA kernels.  There is no fallback: if the shared library is
missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhyena_b200.so")

HYENA_F32, HYENA_BF16 = 0, 1
_DT = {torch.float32: HYENA_F32, torch.bfloat16: HYENA_BF16}

_lock = threading.Lock()
_lib = None

_vp, _fp, _i, _sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_ll, _f = ctypes.c_longlong, ctypes.c_float

# name -> (restype, argtypes)
SIGNATURES = {
    "hyena_status_string": (ctypes.c_char_p, [_i]),
    "hyena_abi_version": (_i, []),
    "hyena_filter_from_modes": (_i, [_fp, _fp, _fp, _i, _i, _i, _fp, _vp]),
    "hyena_filter_spectrum_workspace_bytes": (_sz, [_i, _i, _i]),
    "hyena_filter_spectrum": (_i, [_fp, _i, _i, _i, _fp, _vp, _sz, _vp]),
    "hyena_prefill_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "hyena_prefill_error_offset": (_sz, [_i, _i, _i, _i, _i, _i]),
    "hyena_prefill_uses_tensor_cores": (_i, [_i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "hyena_prefill": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _fp, _fp, _fp, _vp, _fp,
                           _vp, _sz, _vp]),
    "hyena_prefill_chunked_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "hyena_prefill_chunked_error_offset": (_sz, [_i, _i, _i, _i, _i]),
    "hyena_prefill_chunked": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _fp, _fp, _fp, _vp, _fp,
                                   _vp, _sz, _vp]),
    "hyena_prefill_chunked_layers_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "hyena_prefill_chunked_layers_error_offset": (_sz, [_i, _i, _i, _i, _i, _i]),
    "hyena_prefill_chunked_layers": (_i, [_i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                          _vp, _sz, _vp]),
    "hyena_prefill_noalloc_capacity": (_sz, []),
    "hyena_prefill_noalloc": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _fp, _fp, _fp, _vp, _fp,
                                   _vp]),
    "hyena_test_chunked_inject": (_i, [_i, ctypes.c_double]),
    "hyena_test_fail_next_launches": (_i, [_i]),
    "hyena_test_fft_tensor_cores": (_i, [_i]),
    "hyena_debug_bounds_check": (_i, [_vp]),
    "hyena_prompt_state_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "hyena_prompt_state": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _fp, _fp, _vp, _sz, _vp]),
    "hyena_decode_step": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _fp, _fp, _fp, _fp, _vp, _vp]),
    "hyena_decode_step_layers": (_i, [_i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                      _vp]),
    "hyena_fir_cache_prompt": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _fp, _vp]),
    "hyena_fir_decode_step": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _fp, _fp, _vp, _vp]),
    "hyena_linattn_prefill_workspace_bytes": (_sz, [_i] * 7),
    "hyena_linattn_prefill_error_offset": (_sz, [_i] * 7),
    "hyena_linattn_prefill_uses_tensor_cores": (_i, [_i] * 7 + [_ll] * 3 + [_vp] * 4),
    "hyena_test_linattn_hold": (_i, [_i]),
    "hyena_linattn_prefill": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _ll, _ll, _ll, _fp, _f, _vp, _fp, _vp, _fp,
                                   _vp, _sz, _vp]),
    "hyena_linattn_decode_step": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _ll, _ll, _ll, _fp, _f, _vp, _vp, _i, _fp,
                                       _vp, _vp]),
    "hyena_qk_norm_rotate": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _ll, _ll, _vp, _vp, _i, _vp, _vp, _ll, _ll, _vp]),
    "hyena_modal_truncate": (_i, [_fp, _fp, _i, _i, _i, _vp, _fp, _fp, _vp, _vp, _vp]),
}


class HyenaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")
        self.status = status


def _load(path: str):
    if not os.path.exists(path):
        raise RuntimeError(
            f"{os.path.basename(path)} not found at {path}; build it with "
            "`python -m distilled_ssm_decode_b200.build` (there is no CPU fallback)")
    L = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


def lib():
    """The loaded ctypes library (raises if the CUDA library is missing)."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = _load(LIB_PATH)
    return _lib


@contextlib.contextmanager
def using_library(path: str):
    """Route every call of this module through another build of the library (for instance the
    bounds-checked libhyena_b200_dbg.so) inside the `with` block."""
    global _lib
    other = _load(path)
    with _lock:
        prev = _lib
        _lib = other
    linattn_prefill_workspace_bytes.cache_clear()        # the looked-up sizes are another build's
    try:
        yield other
    finally:
        with _lock:
            _lib = prev
        linattn_prefill_workspace_bytes.cache_clear()


def bounds_check():
    """Bounds-checked build only: (status, record) of the first global access out of range since
    the last check; status 0 = none, 1 = record = (file id, source line, index, extent)."""
    rec = (ctypes.c_longlong * 4)()
    st = lib().hyena_debug_bounds_check(ctypes.cast(rec, ctypes.c_void_p))
    return st, tuple(rec)


def status_string(status: int) -> str:
    return lib().hyena_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise HyenaError(fn, status)


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _cuda(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _params(lam, R, Dskip):
    lam = _cuda(lam, "lam", torch.float32)
    R = _cuda(R, "R", torch.float32)
    Dskip = _cuda(Dskip, "Dskip", torch.float32)
    if lam.dim() != 3 or lam.shape[-1] != 2 or R.shape != lam.shape or Dskip.shape != lam.shape[:1]:
        raise ValueError("lam, R must be [H][d][2] float32 and Dskip [H]")
    return lam, R, Dskip


def _act_dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"activations must be float32 or bfloat16, got {t.dtype}")
    return _DT[t.dtype]


# ------------------------------------------------------------------ operations
def filter_from_modes(lam, R, Dskip, L: int) -> torch.Tensor:
    """h [H][L] float32: h_0 = Dskip, h_j = Re sum_n R_n lam_n^(j-1)."""
    lam, R, Dskip = _params(lam, R, Dskip)
    H, d = lam.shape[0], lam.shape[1]
    h = torch.empty((H, L), dtype=torch.float32, device=lam.device)
    _check("hyena_filter_from_modes",
           lib().hyena_filter_from_modes(_ptr(lam), _ptr(R), _ptr(Dskip), H, d, L, _ptr(h),
                                         _stream(lam.device)))
    return h


def filter_spectrum(h, fft_len: int) -> torch.Tensor:
    """complex64 [H][fft_len/2+1]: DFT of each row of h zero-padded to fft_len."""
    h = _cuda(h, "h", torch.float32)
    H, L = h.shape
    out = torch.empty((H, fft_len // 2 + 1, 2), dtype=torch.float32, device=h.device)
    nbytes = lib().hyena_filter_spectrum_workspace_bytes(H, L, fft_len)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=h.device)
    _check("hyena_filter_spectrum",
           lib().hyena_filter_spectrum(_ptr(h), H, L, fft_len, _ptr(out), _ptr(ws), nbytes,
                                       _stream(h.device)))
    return torch.view_as_complex(out)


def prefill_workspace_bytes(B, L, Dch, H, d, fft_len) -> int:
    return int(lib().hyena_prefill_workspace_bytes(B, L, Dch, H, d, fft_len))


def prefill(q, k, v, lam, R, Dskip, fft_len: int, y=None, state=None, workspace=None):
    """FFT prefill.  q,k,v [B][L][Dch] -> (y [B][L][Dch], state float32 [B][d][Dch][2])."""
    lam, R, Dskip = _params(lam, R, Dskip)
    q, k, v = _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v")
    dt = _act_dtype(q)
    B, L, Dch = q.shape
    H, d = lam.shape[0], lam.shape[1]
    if y is None:
        y = torch.empty_like(q)
    if state is None:
        state = torch.empty((B, d, Dch, 2), dtype=torch.float32, device=q.device)
    nbytes = prefill_workspace_bytes(B, L, Dch, H, d, fft_len)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check("hyena_prefill",
           lib().hyena_prefill(_ptr(q), _ptr(k), _ptr(v), dt, B, L, Dch, H, d, fft_len,
                               _ptr(lam), _ptr(R), _ptr(Dskip), _ptr(y), _ptr(state),
                               _ptr(workspace), workspace.numel(), _stream(q.device)))
    return y, state


def prefill_chunked_workspace_bytes(B, L, Dch, H, d) -> int:
    return int(lib().hyena_prefill_chunked_workspace_bytes(B, L, Dch, H, d))


def prefill_chunked(q, k, v, lam, R, Dskip, y=None, state=None, workspace=None):
    """Chunked tensor-core prefill.  q,k,v bf16 [B][L][Dch] -> (y, state [B][d][Dch][2]).

    Returns (y, state, workspace); the int32 at chunked_error_offset() of the
    workspace is 0 after a successful run."""
    lam, R, Dskip = _params(lam, R, Dskip)
    q, k, v = _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v")
    dt = _act_dtype(q)
    B, L, Dch = q.shape
    H, d = lam.shape[0], lam.shape[1]
    if y is None:
        y = torch.empty_like(q)
    if state is None:
        state = torch.empty((B, d, Dch, 2), dtype=torch.float32, device=q.device)
    nbytes = prefill_chunked_workspace_bytes(B, L, Dch, H, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check("hyena_prefill_chunked",
           lib().hyena_prefill_chunked(_ptr(q), _ptr(k), _ptr(v), dt, B, L, Dch, H, d, _ptr(lam),
                                       _ptr(R), _ptr(Dskip), _ptr(y), _ptr(state), _ptr(workspace),
                                       workspace.numel(), _stream(q.device)))
    return y, state, workspace


class PrefillLayerSet:
    """Host pointer arrays of a fixed set of layers for prefill_chunked_layers (built once, so that
    a call costs one library call): per layer q, k, v, y [B][L][Dch] bf16, state [B][d][Dch][2]
    float32 and the modal parameters."""

    def __init__(self, qs, ks, vs, ys, states, lams, Rs, Dskips):
        n = len(qs)
        if not all(len(x) == n for x in (ks, vs, ys, states, lams, Rs, Dskips)):
            raise ValueError("one tensor of each kind per layer")
        q0 = _cuda(qs[0], "q")
        self.dt = _act_dtype(q0)
        self.B, self.L, self.Dch = q0.shape
        ps = [_params(l, r, dk) for l, r, dk in zip(lams, Rs, Dskips)]
        self.H, self.d = ps[0][0].shape[0], ps[0][0].shape[1]
        for name, ts in (("q", qs), ("k", ks), ("v", vs), ("y", ys)):
            for t in ts:
                _cuda(t, name, q0.dtype)
                if tuple(t.shape) != (self.B, self.L, self.Dch):
                    raise ValueError(f"{name}: every layer's tensor must be [B][L][Dch]")
        for st in states:
            _cuda(st, "state", torch.float32)
        if any(p[0].shape != ps[0][0].shape for p in ps):
            raise ValueError("all layers need the same H and d")
        self.n = n
        self._keep = (list(qs), list(ks), list(vs), list(ys), list(states), ps)
        arr = ctypes.c_void_p * max(n, 1)
        self.q, self.k, self.v, self.y, self.state = (arr(*[t.data_ptr() for t in ts]) for ts in (qs, ks, vs, ys, states))
        self.lam = arr(*[p[0].data_ptr() for p in ps])
        self.R = arr(*[p[1].data_ptr() for p in ps])
        self.Dskip = arr(*[p[2].data_ptr() for p in ps])
        self.device = q0.device

    def workspace_bytes(self) -> int:
        return int(lib().hyena_prefill_chunked_layers_workspace_bytes(self.n, self.B, self.L, self.Dch, self.H, self.d))

    def error(self, workspace) -> int:
        """The kernel's error word (synchronises): 0 when every bounded wait succeeded."""
        off = int(lib().hyena_prefill_chunked_layers_error_offset(self.n, self.B, self.L, self.Dch, self.H, self.d))
        return int(workspace[off:off + 4].view(torch.int32).item())


def prefill_chunked_layers(layers: PrefillLayerSet, workspace=None):
    """Chunked prefill of every layer of the set in one launch (writes each layer's y and state).
    Returns the workspace."""
    nbytes = layers.workspace_bytes()
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=layers.device)
    _check("hyena_prefill_chunked_layers",
           lib().hyena_prefill_chunked_layers(layers.n, layers.q, layers.k, layers.v, layers.dt, layers.B, layers.L,
                                              layers.Dch, layers.H, layers.d, layers.lam, layers.R, layers.Dskip,
                                              layers.y, layers.state, _ptr(workspace), workspace.numel(),
                                              _stream(layers.device)))
    return workspace


def chunked_error(workspace, B, L, Dch, H, d) -> int:
    """The kernel's error word (synchronises): 0 when every bounded wait succeeded."""
    off = int(lib().hyena_prefill_chunked_error_offset(B, L, Dch, H, d))
    return int(workspace[off:off + 4].view(torch.int32).item())


def prefill_uses_tensor_cores(q, k, v, H: int, d: int, fft_len: int, y=None) -> bool:
    """Whether prefill(q, k, v, ...) with these tensors runs its transforms on the tensor cores."""
    B, L, Dch = q.shape
    st = lib().hyena_prefill_uses_tensor_cores(_act_dtype(q), B, L, Dch, H, d, fft_len, _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(q if y is None else y))
    if st < 0:
        _check("hyena_prefill_uses_tensor_cores", st)
    return st == 1


def prefill_error(workspace, B, L, Dch, H, d, fft_len) -> int:
    """Error word of the FFT prefill's tensor-core route (synchronises): 0 when its bounded
    waits all succeeded (and always 0 after a call that took the CUDA-core route)."""
    off = int(lib().hyena_prefill_error_offset(B, L, Dch, H, d, fft_len))
    return int(workspace[off:off + 4].view(torch.int32).item())


@contextlib.contextmanager
def fft_tensor_cores(enable: bool):
    """Test hook: inside the block every FFT prefill call runs its transforms on the tensor
    cores where that route applies (enable=True, the default outside) or on the CUDA cores
    only (enable=False)."""
    _check("hyena_test_fft_tensor_cores", lib().hyena_test_fft_tensor_cores(1 if enable else 0))
    try:
        yield
    finally:
        _check("hyena_test_fft_tensor_cores", lib().hyena_test_fft_tensor_cores(1))


def test_chunked_inject(suppress_item: int = -1, lookback_limit_s: float = 0.0):
    """Test hook: fault injection for the chunked prefill's bounded waits (see hyena.h);
    (-1, 0) restores normal operation."""
    _check("hyena_test_chunked_inject", lib().hyena_test_chunked_inject(int(suppress_item), float(lookback_limit_s)))


def prompt_state(k, v, lam, H: int, state=None):
    """state float32 [B][d][Dch][2] = sum_j lam^(L-1-j) k_j v_j (standalone reduction)."""
    lam = _cuda(lam, "lam", torch.float32)
    k, v = _cuda(k, "k"), _cuda(v, "v")
    dt = _act_dtype(k)
    B, L, Dch = k.shape
    d = lam.shape[1]
    if state is None:
        state = torch.empty((B, d, Dch, 2), dtype=torch.float32, device=k.device)
    nbytes = int(lib().hyena_prompt_state_workspace_bytes(B, L, Dch, d))
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=k.device)
    _check("hyena_prompt_state",
           lib().hyena_prompt_state(_ptr(k), _ptr(v), dt, B, L, Dch, H, d, _ptr(lam), _ptr(state),
                                    _ptr(ws), ws.numel(), _stream(k.device)))
    return state


def decode_step(q, k, v, lam, R, Dskip, state, y=None):
    """One decode step: q,k,v [B][Dch]; state [B][d][Dch][2] updated in place; returns y."""
    lam, R, Dskip = _params(lam, R, Dskip)
    q, k, v = _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v")
    state = _cuda(state, "state", torch.float32)
    dt = _act_dtype(q)
    B, Dch = q.shape
    H, d = lam.shape[0], lam.shape[1]
    if y is None:
        y = torch.empty_like(q)
    _check("hyena_decode_step",
           lib().hyena_decode_step(_ptr(q), _ptr(k), _ptr(v), dt, B, Dch, H, d, _ptr(lam), _ptr(R),
                                   _ptr(Dskip), _ptr(state), _ptr(y), _stream(q.device)))
    return y


class LayerSet:
    """Host pointer arrays of a fixed set of layers for decode_step_layers (built once, reused
    every step so that a step costs one library call)."""

    def __init__(self, lams, Rs, Dskips, states):
        n = len(lams)
        if not (len(Rs) == len(Dskips) == len(states) == n):
            raise ValueError("one lam, R, Dskip and state per layer")
        ps = [_params(l, r, dk) for l, r, dk in zip(lams, Rs, Dskips)]
        self.H, self.d = ps[0][0].shape[0], ps[0][0].shape[1]
        if any(p[0].shape != ps[0][0].shape for p in ps):
            raise ValueError("all layers need the same H and d")
        self.states = [_cuda(s, "state", torch.float32) for s in states]
        self.n = n
        arr = ctypes.c_void_p * max(n, 1)
        self._keep = ps
        self.lam = arr(*[p[0].data_ptr() for p in ps])
        self.R = arr(*[p[1].data_ptr() for p in ps])
        self.Dskip = arr(*[p[2].data_ptr() for p in ps])
        self.state = arr(*[s.data_ptr() for s in self.states])


def decode_step_layers(layers: LayerSet, qs, ks, vs, ys):
    """One decode step of every layer in one launch: qs[i], ks[i], vs[i], ys[i] [B][Dch] for
    layer i; each layer's state is updated in place.  qs..ys are sequences of tensors, or
    [layers][B][Dch] tensors."""
    n = layers.n
    arr = ctypes.c_void_p * max(n, 1)
    q0 = _cuda(qs[0], "q")
    dt = _act_dtype(q0)
    B, Dch = q0.shape
    for name, ts in (("q", qs), ("k", ks), ("v", vs), ("y", ys)):
        if len(ts) != n:
            raise ValueError(f"{name}: one tensor per layer")
        for t in ts:
            _cuda(t, name, q0.dtype)
            if tuple(t.shape) != (B, Dch):
                raise ValueError(f"{name}: every layer's tensor must be [B][Dch]")
    pq, pk, pv, py = (arr(*[t.data_ptr() for t in ts]) for ts in (qs, ks, vs, ys))
    _check("hyena_decode_step_layers",
           lib().hyena_decode_step_layers(n, pq, pk, pv, dt, B, Dch, layers.H, layers.d, layers.lam,
                                          layers.R, layers.Dskip, layers.state, py,
                                          _stream(q0.device)))
    return ys


def fir_cache_prompt(k, v, t_max: int, u_cache=None):
    """History of a prompt for the undistilled baseline: u_cache float32 [B][t_max][Dch] with
    rows j < L set to k_j v_j (the rest left as they are)."""
    k, v = _cuda(k, "k"), _cuda(v, "v")
    dt = _act_dtype(k)
    B, L, Dch = k.shape
    if u_cache is None:
        u_cache = torch.zeros((B, t_max, Dch), dtype=torch.float32, device=k.device)
    _cuda(u_cache, "u_cache", torch.float32)
    _check("hyena_fir_cache_prompt",
           lib().hyena_fir_cache_prompt(_ptr(k), _ptr(v), dt, B, L, Dch, t_max, _ptr(u_cache),
                                        _stream(k.device)))
    return u_cache


def fir_decode_step(q, k, v, h, u_cache, t: int, y=None):
    """Undistilled decode of token t: y = q (sum_{j<=t} h_{t-j} u_j), history in u_cache
    [B][t_max][Dch] (row t is written); h [H][t_max] float32 taps."""
    q, k, v = _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v")
    h = _cuda(h, "h", torch.float32)
    u_cache = _cuda(u_cache, "u_cache", torch.float32)
    dt = _act_dtype(q)
    B, Dch = q.shape
    H, t_max = h.shape
    if u_cache.shape != (B, t_max, Dch):
        raise ValueError("u_cache must be [B][t_max][Dch] with t_max = h.shape[1]")
    if y is None:
        y = torch.empty_like(q)
    _check("hyena_fir_decode_step",
           lib().hyena_fir_decode_step(_ptr(q), _ptr(k), _ptr(v), dt, B, Dch, H, t, t_max, _ptr(h),
                                       _ptr(u_cache), _ptr(y), _stream(q.device)))
    return y


def modal_truncate(lam, R, k: int):
    """Keep the k modes of largest |R|/(1-|lambda|) per head.  Returns (kept int32 [H][k],
    lam_out, R_out float32 [H][k][2], bound float64 [H], err_l2 float64 [H])."""
    lam = _cuda(lam, "lam", torch.float32)
    R = _cuda(R, "R", torch.float32)
    H, d = lam.shape[0], lam.shape[1]
    dev = lam.device
    kept = torch.empty((H, k), dtype=torch.int32, device=dev)
    lo = torch.empty((H, k, 2), dtype=torch.float32, device=dev)
    ro = torch.empty((H, k, 2), dtype=torch.float32, device=dev)
    bound = torch.empty(H, dtype=torch.float64, device=dev)
    err = torch.empty(H, dtype=torch.float64, device=dev)
    nul = lambda t: _ptr(t) if k > 0 else None
    _check("hyena_modal_truncate",
           lib().hyena_modal_truncate(_ptr(lam), _ptr(R), H, d, k, nul(kept), nul(lo), nul(ro), _ptr(bound),
                                      _ptr(err), _stream(dev)))
    return kept, lo, ro, bound, err



# ------------------------------------------------------------------ linear attention
# A token's step takes a few microseconds on the GPU, so the host side of these calls is kept short: pointers go
# to ctypes as plain integers, the stream is read as a number, sizes of workspaces are looked up.
_INT_MAX = 0x7fffffff     # the library's sizes and positions; ctypes would cut larger ones to their low bits


def _rows(t: torch.Tensor, name: str, dim: int, dtype, device):
    """Row stride (elements between consecutive tokens) of q, k or v [B][L][heads][width] (dim 4) or
    [B][heads][width] (dim 3): heads and width contiguous, rows evenly spaced, as a slice of one
    projection's output has them."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    sh, st = t.shape, t.stride()
    if len(sh) != dim:
        raise ValueError(f"{name} must have {dim} dimensions")
    if t.numel() > _INT_MAX and max(sh) > _INT_MAX:
        raise ValueError(f"{name}: sizes must fit 32 bits, got {list(sh)}")
    if dim == 3:
        rows, heads, width = sh
        s_row, s_head, s_entry = st
        tokens, s_token = 1, 0
    else:
        rows, tokens, heads, width = sh
        s_row, s_token, s_head, s_entry = st
    n = heads * width
    if n == 0 or rows == 0 or tokens == 0:
        return n
    if (s_entry != 1 and width > 1) or (s_head != width and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if tokens == 1:
        ld = s_row if rows > 1 else n
    else:
        ld = s_token
        if rows > 1 and s_row != tokens * ld:
            raise ValueError(f"{name}: batch rows must follow each other at the token stride")
    if ld < n:
        raise ValueError(f"{name}: tokens overlap")
    return ld


def _plain(t, name: str, dtype, shape, device):
    """The address of a contiguous tensor of this dtype, shape and device (None: None)."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _cuda(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t.data_ptr()


def _position(pos0):
    if not -_INT_MAX - 1 <= pos0 <= _INT_MAX:
        raise ValueError(f"pos0 must fit 32 bits, got {pos0}")
    return pos0


def _run(fn: str, device, *args):
    """Call a library function on the current stream of `device` (the library works on the current device)."""
    f = getattr(_lib or lib(), fn)
    if torch.cuda.current_device() == device.index:
        st = f(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            st = f(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if st != 0:
        raise HyenaError(fn, st)


class _CQKPrep(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int), ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("inv_freq", ctypes.c_void_p),
                ("interleaved", ctypes.c_int)]


class QKPrep:
    """What qk_norm_rotate does to each head of the queries and keys (keep one beside the weights).

    wq, wk: float32 [hd] norm weights (None: ones); eps inside the square root; norm=False leaves
    the norm out.  inv_freq: float32 [rot_dim / 2], the angle per position of each pair (None: no
    rotation); interleaved pairs are (2i, 2i+1), else (i, i + rot_dim / 2)."""

    def __init__(self, wq=None, wk=None, eps: float = 1e-6, inv_freq=None, interleaved: bool = False, norm: bool = True):
        for name, t in (("wq", wq), ("wk", wk), ("inv_freq", inv_freq)):
            if t is not None and _cuda(t, name, torch.float32).dim() != 1:
                raise ValueError(f"{name} must have one dimension")
        self.wq, self.wk, self.inv_freq = wq, wk, inv_freq
        self.rot_dim = 0 if inv_freq is None else 2 * inv_freq.numel()
        at = lambda t: t.data_ptr() if t is not None and t.numel() else None
        self._c = _CQKPrep(int(norm), eps, at(wq), at(wk), self.rot_dim, at(inv_freq), int(interleaved))
        self._ref = ctypes.c_void_p(ctypes.addressof(self._c))

    def _check(self, hd: int, device):
        for name, t in (("wq", self.wq), ("wk", self.wk)):
            if t is not None and (t.numel() != hd or t.device != device):
                raise ValueError(f"{name} must be [{hd}] on {device}")
        if self.inv_freq is not None and self.inv_freq.device != device:
            raise ValueError(f"inv_freq must be on {device}")
        return self._ref


def qk_norm_rotate(q, k, prep: QKPrep, positions=None, pos0: int = 0, q_out=None, k_out=None):
    """Norm of each head of q [B][L][H][hd] and k [B][L][Hk][hd], and the position rotation, in one
    pass.  positions int32 [B][L], or None: token t stands at pos0 + t.  q_out=q, k_out=k work in
    place.  Returns (q_out, k_out)."""
    dt, dev = _act_dtype(q), q.device
    dtype = q.dtype
    ldq, ldk = _rows(q, "q", 4, dtype, dev), _rows(k, "k", 4, dtype, dev)
    B, L, H, hd = q.shape
    Bk, Lk, Hk, hk = k.shape
    if Bk != B or Lk != L or hk != hd:
        raise ValueError("q and k must be [B][L][heads][hd] with the same B, L and hd")
    pos = _plain(positions, "positions", torch.int32, (B, L), dev)
    ldqo, ldko = H * hd, Hk * hd
    if q_out is None:
        q_out = q.new_empty((B, L, H, hd))
    else:
        ldqo = _rows(q_out, "q_out", 4, dtype, dev)
    if k_out is None:
        k_out = k.new_empty((B, L, Hk, hd))
    else:
        ldko = _rows(k_out, "k_out", 4, dtype, dev)
    if q_out.shape != q.shape or k_out.shape != k.shape:
        raise ValueError("q_out and k_out must have the shapes of q and k")
    _run("hyena_qk_norm_rotate", dev, q.data_ptr(), k.data_ptr(), dt, B, L, H, Hk, hd, ldq, ldk, prep._check(hd, dev),
         pos, _position(pos0), q_out.data_ptr(), k_out.data_ptr(), ldqo, ldko)
    return q_out, k_out


@functools.lru_cache(maxsize=4096)
def linattn_prefill_workspace_bytes(dtype, B, L, H, Hk, dk, dv) -> int:
    return int(lib().hyena_linattn_prefill_workspace_bytes(_DT[dtype], B, L, H, Hk, dk, dv))


class LinattnPrefill(tuple):
    """(o, state) of linattn_prefill, which unpacks as the two tensors, with the call's workspace.  On the
    tensor-core route the results hold only if error() is 0: its bounded waits report there."""

    def __new__(cls, o, state, workspace, dims):
        self = super().__new__(cls, (o, state))
        self.workspace, self._dims = workspace, dims
        return self

    def __reduce__(self):
        return tuple, (tuple(self),)          # copies are of the two tensors alone

    def error(self) -> int:
        """0 when the call's every bounded wait succeeded (synchronises; before the workspace is used again)."""
        return linattn_error(self.workspace, *self._dims)


def linattn_prefill(q, k, v, decay, scale: float = 1.0, lens=None, state_in=None, o=None, state=None, workspace=None):
    """Linear attention with a decay for each head over a prompt: S_t = g S_{t-1} + k_t v_t^T,
    o_t = scale S_t^T q_t.

    q [B][L][H][dk], k [B][L][Hk][dk], v [B][L][Hk][dv] (slices of one projection work), decay float32
    [Hk], lens int32 [B] (tokens of each row; the rows of o behind them are left as they were, zero
    if o is made here), state_in float32 [B][Hk][dk][dv].  Returns (o [B][L][H][dv], state), a
    LinattnPrefill: its error() is 0 once the call has run, unless a bounded wait gave up and the results are
    not valid."""
    dt, dev = _act_dtype(q), q.device
    dtype = q.dtype
    ldq, ldk, ldv = _rows(q, "q", 4, dtype, dev), _rows(k, "k", 4, dtype, dev), _rows(v, "v", 4, dtype, dev)
    B, L, H, dk = q.shape
    Bv, Lv, Hk, dv = v.shape
    if k.shape != (B, L, Hk, dk) or Bv != B or Lv != L:
        raise ValueError("q [B][L][H][dk], k [B][L][Hk][dk], v [B][L][Hk][dv] expected")
    sshape = (B, Hk, dk, dv)
    decay_at = _plain(decay, "decay", torch.float32, (Hk,), dev)
    lens_at = _plain(lens, "lens", torch.int32, (B,), dev)
    in_at = _plain(state_in, "state_in", torch.float32, sshape, dev)
    if o is None:
        o = (q.new_empty if lens is None else q.new_zeros)((B, L, H, dv))
    if state is None:
        state = q.new_empty(sshape, dtype=torch.float32)
    o_at = _plain(o, "o", dtype, (B, L, H, dv), dev)
    state_at = _plain(state, "state", torch.float32, sshape, dev)
    if workspace is None:
        workspace = q.new_empty(max(linattn_prefill_workspace_bytes(dtype, B, L, H, Hk, dk, dv), 1), dtype=torch.uint8)
    _cuda(workspace, "workspace", torch.uint8)
    if workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}, got {workspace.device}")
    _run("hyena_linattn_prefill", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, B, L, H, Hk, dk, dv, ldq, ldk, ldv,
         decay_at, scale, lens_at, in_at, o_at, state_at, workspace.data_ptr(), workspace.numel())
    return LinattnPrefill(o, state, workspace, (dtype, B, L, H, Hk, dk, dv))


def linattn_prefill_uses_tensor_cores(q, k, v, o=None) -> bool:
    """Whether linattn_prefill with these tensors runs on the tensor cores (o None: a new one)."""
    B, L, H, dk = q.shape
    Hk, dv = v.shape[2:]
    ld = [_rows(t, n, 4, q.dtype, q.device) for t, n in ((q, "q"), (k, "k"), (v, "v"))]
    st = lib().hyena_linattn_prefill_uses_tensor_cores(_act_dtype(q), B, L, H, Hk, dk, dv, *ld, _ptr(q), _ptr(k), _ptr(v),
                                                      _ptr(o))
    if st < 0:
        _check("hyena_linattn_prefill_uses_tensor_cores", st)
    return st == 1


def linattn_error(workspace, dtype, B, L, H, Hk, dk, dv) -> int:
    """The error words of linattn_prefill (synchronises): 0 when every bounded wait succeeded."""
    if B == 0 or L == 0:
        return 0            # nothing ran
    lo = int(lib().hyena_linattn_prefill_error_offset(_DT[dtype], B, L, H, Hk, dk, dv))
    hi = linattn_prefill_workspace_bytes(dtype, B, L, H, Hk, dk, dv)
    return int(workspace[lo:hi].view(torch.int32).abs().max().item())


@contextlib.contextmanager
def linattn_hold():
    """Test hook: inside the block a bounded wait of every tensor-core linattn_prefill runs out (see
    hyena.h)."""
    _check("hyena_test_linattn_hold", lib().hyena_test_linattn_hold(1))
    try:
        yield
    finally:
        _check("hyena_test_linattn_hold", lib().hyena_test_linattn_hold(0))


def linattn_decode_step(q, k, v, decay, state, scale: float = 1.0, prep: QKPrep = None, positions=None, pos0: int = 0,
                        o=None):
    """One token: S <- g S + k v^T (state [B][Hk][dk][dv] in place), o = scale S^T q.

    q [B][H][dk], k [B][Hk][dk], v [B][Hk][dv] (slices of one projection work).  With prep, q and k pass
    through qk_norm_rotate's formulas in the same launch, at positions int32 [B] (None: pos0).
    Returns o [B][H][dv]."""
    dt, dev = _act_dtype(q), q.device
    dtype = q.dtype
    ldq, ldk, ldv = _rows(q, "q", 3, dtype, dev), _rows(k, "k", 3, dtype, dev), _rows(v, "v", 3, dtype, dev)
    B, H, dk = q.shape
    Bv, Hk, dv = v.shape
    if k.shape != (B, Hk, dk) or Bv != B:
        raise ValueError("q [B][H][dk], k [B][Hk][dk], v [B][Hk][dv] expected")
    if state is None:
        raise TypeError("state must be a CUDA tensor")
    decay_at = _plain(decay, "decay", torch.float32, (Hk,), dev)
    state_at = _plain(state, "state", torch.float32, (B, Hk, dk, dv), dev)
    pos = _plain(positions, "positions", torch.int32, (B,), dev)
    if o is None:
        o = q.new_empty((B, H, dv))
        o_at = o.data_ptr()
    else:
        o_at = _plain(o, "o", dtype, (B, H, dv), dev)
    _run("hyena_linattn_decode_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, B, H, Hk, dk, dv, ldq, ldk, ldv,
         decay_at, scale, None if prep is None else prep._check(dk, dev), pos, _position(pos0), state_at, o_at)
    return o
