"""ctypes binding of libsvlinattn.so: argument marshalling only, every step runs in the library.

Functions carry the C entry points' names. Tensors are torch CUDA tensors (PyTorch supplies device
memory and streams); outputs and the workspace are allocated here when the caller gives none.
There is no fallback: if the shared library is missing or the device is not a B200 the call
raises.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsvlinattn.so")
_lib = None
_lock = threading.Lock()

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_UNSUPPORTED, SV_ERR_CUDA, SV_ERR_TIMEOUT = range(5)
SV_BF16, SV_F32 = 0, 1
SV_MXFP8, SV_MXFP4, SV_NVFP4 = range(3)
SV_OP_LINATTN_FWD, SV_OP_BLOCK_STATE_UPDATE, SV_OP_BLOCK_CAUSAL_ATTN, SV_OP_CACHE_STEP = range(4)

#: every symbol include/svlinattn.h declares
EXPORTS = (
    "sv_workspace_bytes", "sv_workspace_init", "sv_device_status", "sv_workspace_set_mirror", "sv_linattn_fwd",
    "sv_block_state_update", "sv_block_causal_attn", "sv_cache_step", "sv_cache_step_noalloc",
    "sv_cache_step_noalloc_status", "sv_temporal_conv", "sv_temporal_conv_step", "sv_qkv_projection",
    "sv_out_projection", "sv_mx_code_bytes", "sv_mx_scale_bytes", "sv_mx_global_scale", "sv_mx_quantize",
    "sv_mx_dequantize", "sv_rmsnorm", "sv_mx_projection", "sv_mx_qkv_projection", "sv_rope3d_table_bytes", "sv_rope3d_table", "sv_block_causal_attn_rope", "sv_profile_events",
    "sv_last_error", "sv_selftest_wait_timeout", "sv_version",
)


class SvRope3d(ctypes.Structure):
    """The C descriptor sv_rope3d (include/svlinattn.h)."""

    _fields_ = [("table", ctypes.c_void_p), ("frames", ctypes.c_int), ("height", ctypes.c_int),
                ("width", ctypes.c_int), ("D", ctypes.c_int), ("pairs_t", ctypes.c_int), ("pairs_h", ctypes.c_int),
                ("pairs_w", ctypes.c_int), ("frame0", ctypes.c_int)]


class SvMx(ctypes.Structure):
    """The C descriptor sv_mx (include/svlinattn.h)."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("gscale", ctypes.c_void_p),
                ("rows", ctypes.c_longlong), ("cols", ctypes.c_int), ("fmt", ctypes.c_int)]


class SvError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"sv status {status}: {msg}")
        self.status = status


def lib_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load libsvlinattn.so (built in-tree by block_causal_linear_relu_b200.build)."""
    global _lib
    if _lib is not None:  # loaded: no lock on the per-call path
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with `python -m block_causal_linear_relu_b200.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, sz, i, f, u32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float, ctypes.POINTER(ctypes.c_uint32)
        lib.sv_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
        lib.sv_workspace_bytes.restype = sz
        lib.sv_workspace_init.argtypes = [vp, sz, vp]
        lib.sv_workspace_init.restype = i
        lib.sv_device_status.argtypes = [vp, vp, u32p]
        lib.sv_device_status.restype = i
        lib.sv_workspace_set_mirror.argtypes = [vp, sz, vp, vp]
        lib.sv_workspace_set_mirror.restype = i
        lib.sv_linattn_fwd.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, vp, sz, vp]
        lib.sv_linattn_fwd.restype = i
        lib.sv_block_state_update.argtypes = [vp, vp, i, i, i, i, i, vp, vp, vp, sz, vp]
        lib.sv_block_state_update.restype = i
        lib.sv_block_causal_attn.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, vp, vp, vp, vp, vp, sz, vp]
        lib.sv_block_causal_attn.restype = i
        lib.sv_cache_step.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, vp, vp, i, vp, sz, vp]
        lib.sv_cache_step.restype = i
        lib.sv_cache_step_noalloc.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, vp, vp, i, vp]
        lib.sv_cache_step_noalloc.restype = i
        lib.sv_cache_step_noalloc_status.argtypes = [vp, u32p]
        lib.sv_cache_step_noalloc_status.restype = i
        lib.sv_temporal_conv.argtypes = [vp, vp, i, i, i, i, i, vp, vp, i, vp]
        lib.sv_temporal_conv.restype = i
        lib.sv_temporal_conv_step.argtypes = [vp, vp, i, i, i, i, vp, vp, vp, i, i, vp]
        lib.sv_temporal_conv_step.restype = i
        lib.sv_qkv_projection.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, vp, sz, vp]
        lib.sv_qkv_projection.restype = i
        lib.sv_out_projection.argtypes = [vp, vp, vp, i, i, i, i, i, vp, sz, vp]
        lib.sv_out_projection.restype = i
        ll, mx = ctypes.c_longlong, ctypes.POINTER(SvMx)
        lib.sv_mx_code_bytes.argtypes = [i, ll, i]
        lib.sv_mx_code_bytes.restype = sz
        lib.sv_mx_scale_bytes.argtypes = [i, ll, i]
        lib.sv_mx_scale_bytes.restype = sz
        lib.sv_mx_global_scale.argtypes = [vp, ll, i, vp, vp]
        lib.sv_mx_global_scale.restype = i
        lib.sv_mx_quantize.argtypes = [vp, i, i, i, i, i, mx, vp]
        lib.sv_mx_quantize.restype = i
        lib.sv_mx_dequantize.argtypes = [mx, vp, i, vp]
        lib.sv_mx_dequantize.restype = i
        lib.sv_rmsnorm.argtypes = [vp, vp, vp, vp, ll, i, i, f, vp, mx, vp]
        lib.sv_rmsnorm.restype = i
        lib.sv_mx_projection.argtypes = [mx, mx, vp, vp, sz, vp]
        lib.sv_mx_projection.restype = i
        lib.sv_mx_qkv_projection.argtypes = [mx, mx, vp, vp, vp, i, i, i, i, vp, sz, vp]
        lib.sv_mx_qkv_projection.restype = i
        lib.sv_rope3d_table_bytes.argtypes = [i, i, i, i]
        lib.sv_rope3d_table_bytes.restype = sz
        lib.sv_rope3d_table.argtypes = [vp, sz, i, i, i, i, i, i, i, f, vp]
        lib.sv_rope3d_table.restype = i
        lib.sv_block_causal_attn_rope.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, vp, vp, vp, vp,
                                                  ctypes.POINTER(SvRope3d), vp, sz, vp]
        lib.sv_block_causal_attn_rope.restype = i
        lib.sv_profile_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), i]
        lib.sv_profile_events.restype = i
        lib.sv_last_error.argtypes = []
        lib.sv_last_error.restype = ctypes.c_char_p
        lib.sv_selftest_wait_timeout.argtypes = [vp, sz, vp]
        lib.sv_selftest_wait_timeout.restype = i
        lib.sv_version.argtypes = []
        lib.sv_version.restype = i
        _lib = lib
        return lib


def _check(status: int):
    if status != SV_OK:
        raise SvError(status, load().sv_last_error().decode())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise TypeError(f"unsupported dtype {t.dtype}: bfloat16 or float32 expected")


def _ptr(t):
    # plain ints (and None) convert to the c_void_p parameters without a ctypes object per call
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _on(stream):
    """Makes `stream` the current one: a torch stream, or any object with a cuda_stream handle."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _empty(stream, dtype, device, *shape):
    """An uninitialised tensor that a call on `stream` (None: the current stream) writes.

    Its memory belongs to the stream that writes it: memory freed on the current stream may still be read or
    written there by queued kernels, which a call on another stream does not wait for. The current stream is
    recorded as one that uses the tensor too, so that it may be read there and dropped without a wait."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with _on(stream):
        t = torch.empty(*shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _empty_like(x, stream):
    return torch.empty_like(x) if stream is None else _empty(stream, x.dtype, x.device, *x.shape)


def _qkv(*ts):
    """Checks q, k, v (and o) in one pass; returns their shape [B, H, N, D]."""
    ref = ts[0]
    shape, dtype, device = ref.shape, ref.dtype, ref.device
    if not ref.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if len(shape) != 4:
        raise ValueError("q, k, v, o must share shape [B, H, N, D], dtype and device")
    for t in ts:
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous [B, H, N, D]")
        if t is not ref and (t.shape != shape or t.dtype != dtype or t.device != device):
            raise ValueError("q, k, v, o must share shape [B, H, N, D], dtype and device")
    return shape


def workspace_bytes(op: int, B: int, H: int, N: int, D: int, block_len: int, dtype: int, device=None) -> int:
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = load().sv_workspace_bytes(op, B, H, N, D, block_len, dtype)
    if n == 0:
        raise SvError(SV_ERR_INVALID_ARG, load().sv_last_error().decode())
    return int(n)


class Workspace:
    """Caller-owned device scratch: a 256-byte aligned view into a torch uint8 buffer.

    A page-locked host word is registered as the workspace's status mirror: a kernel whose bounded
    wait expires writes its status code there as well, so every later call of this binding on the
    workspace raises SvError(SV_ERR_TIMEOUT) before it launches anything (``check``), without a
    synchronisation per call. ``status`` synchronises, reads and clears the device word.
    """

    def __init__(self, nbytes: int, device, stream=None):
        self.buf = _empty(stream, torch.uint8, device, nbytes + 256)
        off = (-self.buf.data_ptr()) % 256
        self.view = self.buf[off:off + nbytes]
        self.nbytes = nbytes
        self._ptr = self.view.data_ptr()
        self._mirror = torch.zeros(1, dtype=torch.int32).pin_memory()
        self._mirror_np = self._mirror.numpy()
        self._word = memoryview(self._mirror_np)  # read before every call: a Python int, not a numpy scalar
        lib = load()
        with torch.cuda.device(self.buf.device):
            _check(lib.sv_workspace_init(self._ptr, nbytes, _stream(stream)))
            _check(lib.sv_workspace_set_mirror(self._ptr, nbytes, self._mirror.data_ptr(), _stream(stream)))

    @property
    def ptr(self):
        return self._ptr

    def status(self, stream=None) -> int:
        """Synchronise, return the device status word (0 = no timeout) and clear it (and the mirror)."""
        code = ctypes.c_uint32(0)
        st = load().sv_device_status(self.ptr, _stream(stream), ctypes.byref(code))
        if st not in (SV_OK, SV_ERR_TIMEOUT):
            _check(st)
        self._mirror_np[0] = 0
        return int(code.value)

    def check(self, stream=None):
        """Raise SvError(SV_ERR_TIMEOUT) if a kernel has reported a timeout on this workspace since the
        last check (reads the host mirror: no synchronisation unless a timeout was reported)."""
        if self._word[0]:
            code = self.status(stream)
            raise SvError(SV_ERR_TIMEOUT, f"a kernel's bounded wait expired on this workspace "
                                          f"(status word 0x{code:08x}); its output was not written")


def sv_selftest_wait_timeout(ws: Workspace, stream=None):
    """Launch the bounded-wait self-test on `ws` (its status word is raised about 2 s later; read it
    with ws.status())."""
    _check(load().sv_selftest_wait_timeout(ws.ptr, ws.nbytes, _stream(stream)))


def make_workspace(op: int, q_like: torch.Tensor, block_len: int | None = None, stream=None) -> Workspace:
    B, H, N, D = q_like.shape
    n = workspace_bytes(op, B, H, N, D, block_len if block_len is not None else N, _dt(q_like), q_like.device)
    return Workspace(n, q_like.device, stream)


_default_ws = {}


def _ws(ws, op, q_like, block_len, stream):
    """The caller's workspace, else one kept per (device, stream, op, sizes), so that calls without
    an explicit workspace reuse it (calls on one stream are ordered) and see its reported timeouts."""
    if ws is None:
        B, H, N, D = q_like.shape
        key = (q_like.device.index, _stream(stream), op, B, H, N, D, block_len, q_like.dtype)
        ws = _default_ws.get(key)
        if ws is None:
            ws = _default_ws[key] = make_workspace(op, q_like, block_len, stream)
    ws.check(stream)
    return ws


def sv_linattn_fwd(q, k, v, o=None, eps: float = 1e-6, ws: Workspace | None = None, stream=None):
    """Bidirectional ReLU linear attention; returns o."""
    o = _empty_like(q, stream) if o is None else o
    B, H, N, D = _qkv(q, k, v, o)
    ws = _ws(ws, SV_OP_LINATTN_FWD, q, None, stream)
    _check(load().sv_linattn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, D, _dt(q), eps, ws.ptr, ws.nbytes,
                                 _stream(stream)))
    return o


def sv_block_causal_attn(q, k, v, block_len: int, o=None, eps: float = 1e-6, S_in=None, z_in=None, S_out=None,
                         z_out=None, ws: Workspace | None = None, stream=None):
    """Block-causal prefill; returns o (S_out/z_out are written in place when given)."""
    o = _empty_like(q, stream) if o is None else o
    B, H, N, D = _qkv(q, k, v, o)
    for t in (S_in, z_in, S_out, z_out):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or t.device != q.device):
            raise ValueError("S/z must be contiguous float32 tensors on q's device")
    ws = _ws(ws, SV_OP_BLOCK_CAUSAL_ATTN, q, block_len, stream)
    _check(load().sv_block_causal_attn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, D, int(block_len), _dt(q), eps,
                                       _ptr(S_in), _ptr(z_in), _ptr(S_out), _ptr(z_out), ws.ptr, ws.nbytes,
                                       _stream(stream)))
    return o


def sv_cache_step(q, k, v, S, z, commit: bool = True, o=None, eps: float = 1e-6, ws: Workspace | None = None,
                  stream=None):
    """One streaming block against the fp32 cache (S [B,H,D,D], z [B,H,D]); returns o."""
    o = _empty_like(q, stream) if o is None else o
    B, H, N, D = _qkv(q, k, v, o)
    if S.dtype != torch.float32 or z.dtype != torch.float32 or tuple(S.shape) != (B, H, D, D) or tuple(z.shape) != (B, H, D):
        raise ValueError("cache must be float32 S [B,H,D,D] and z [B,H,D]")
    ws = _ws(ws, SV_OP_CACHE_STEP, q, None, stream)
    _check(load().sv_cache_step(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, D, _dt(q), eps, _ptr(S), _ptr(z),
                                1 if commit else 0, ws.ptr, ws.nbytes, _stream(stream)))
    return o


def sv_cache_step_noalloc(q, k, v, S, z, commit: bool = True, o=None, eps: float = 1e-6, stream=None):
    """sv_cache_step with the library's static scratch instead of a workspace (see the header)."""
    o = _empty_like(q, stream) if o is None else o
    B, H, N, D = _qkv(q, k, v, o)
    if S.dtype != torch.float32 or z.dtype != torch.float32 or tuple(S.shape) != (B, H, D, D) or tuple(z.shape) != (B, H, D):
        raise ValueError("cache must be float32 S [B,H,D,D] and z [B,H,D]")
    _check(load().sv_cache_step_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, D, _dt(q), eps, _ptr(S),
                                        _ptr(z), 1 if commit else 0, _stream(stream)))
    return o


def sv_cache_step_noalloc_status(stream=None) -> int:
    """Synchronise and return (then clear) the status word of sv_cache_step_noalloc's static scratch
    on the current device (0 = no timeout)."""
    code = ctypes.c_uint32(0)
    st = load().sv_cache_step_noalloc_status(_stream(stream), ctypes.byref(code))
    if st not in (SV_OK, SV_ERR_TIMEOUT):
        _check(st)
    return int(code.value)


def sv_profile_events(events):
    """Install (list of 4 torch.cuda.Event, already recorded once) or clear (None) the timing hook."""
    if events is None:
        _check(load().sv_profile_events(None, 0))
        return
    arr = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(load().sv_profile_events(arr, 4))


def sv_block_state_update(k, v, S, z, ws: Workspace | None = None, stream=None):
    """S += ReLU(K)^T V, z += sum ReLU(k), in place."""
    B, H, N, D = _qkv(k, v)
    if S.dtype != torch.float32 or z.dtype != torch.float32 or tuple(S.shape) != (B, H, D, D) or tuple(z.shape) != (B, H, D):
        raise ValueError("cache must be float32 S [B,H,D,D] and z [B,H,D]")
    ws = _ws(ws, SV_OP_BLOCK_STATE_UPDATE, k, None, stream)
    _check(load().sv_block_state_update(_ptr(k), _ptr(v), B, H, N, D, _dt(k), _ptr(S), _ptr(z), ws.ptr, ws.nbytes,
                                        _stream(stream)))
    return S, z


def _conv_args(x, w, bias):
    if not x.is_cuda or x.dim() != 4 or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor [B, T, S, C]")
    C = x.shape[3]
    if w.dtype != torch.float32 or tuple(w.shape) != (C, 3) or not w.is_contiguous() or w.device != x.device:
        raise ValueError("w must be a contiguous float32 [C, 3] tensor on x's device")
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (C,) or bias.device != x.device):
        raise ValueError("bias must be a float32 [C] tensor on x's device")


def sv_temporal_conv(x, w, frames_per_block: int, bias=None, y=None, stream=None):
    """Block-causal temporal convolution over x [B, T, S, C] (kernel width 3); returns y."""
    _conv_args(x, w, bias)
    y = _empty_like(x, stream) if y is None else y
    B, T, S, C = x.shape
    _check(load().sv_temporal_conv(_ptr(x), _ptr(y), B, T, S, C, int(frames_per_block), _ptr(w), _ptr(bias), _dt(x),
                                   _stream(stream)))
    return y


def sv_temporal_conv_step(x, w, carry, commit: bool = True, bias=None, y=None, stream=None):
    """One block x [B, T, S, C] of a stream with the previous block's last frame in carry [B, S, C]
    (zeros before the first block); carry takes x's last frame if commit. Returns y."""
    _conv_args(x, w, bias)
    B, T, S, C = x.shape
    if carry.dtype != x.dtype or tuple(carry.shape) != (B, S, C) or not carry.is_contiguous():
        raise ValueError("carry must be a contiguous [B, S, C] tensor of x's dtype")
    y = _empty_like(x, stream) if y is None else y
    _check(load().sv_temporal_conv_step(_ptr(x), _ptr(y), B, T, S, C, _ptr(w), _ptr(bias), _ptr(carry),
                                        1 if commit else 0, _dt(x), _stream(stream)))
    return y


_proj_ws = {}


def _proj_workspace(device, stream):
    key = (device.index, _stream(stream))
    ws = _proj_ws.get(key)
    if ws is None:
        ws = _proj_ws[key] = Workspace(256, device, stream)
    ws.check(stream)
    return ws


def sv_qkv_projection(x, w_qkv, H: int, D: int, q=None, k=None, v=None, ws: Workspace | None = None, stream=None):
    """x [B, N, C] bf16, w_qkv [3*H*D, C] bf16 -> (ReLU(q), ReLU(k), v), each [B, H, N, D] bf16."""
    if not x.is_cuda or x.dim() != 3 or x.dtype != torch.bfloat16 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bfloat16 CUDA tensor [B, N, C]")
    B, N, C = x.shape
    if tuple(w_qkv.shape) != (3 * H * D, C) or w_qkv.dtype != torch.bfloat16 or not w_qkv.is_contiguous():
        raise ValueError("w_qkv must be a contiguous bfloat16 [3*H*D, C] tensor")
    q, k, v = (_empty(stream, torch.bfloat16, x.device, B, H, N, D) if t is None else t
               for t in (q, k, v))
    ws = ws if ws is not None else _proj_workspace(x.device, stream)
    _check(load().sv_qkv_projection(_ptr(x), _ptr(w_qkv), _ptr(q), _ptr(k), _ptr(v), B, N, C, H, D, ws.ptr, ws.nbytes,
                                    _stream(stream)))
    return q, k, v


def sv_out_projection(o, w_o, y=None, ws: Workspace | None = None, stream=None):
    """o [B, H, N, D] bf16, w_o [C_out, H*D] bf16 -> y [B, N, C_out] bf16."""
    if not o.is_cuda or o.dim() != 4 or o.dtype != torch.bfloat16 or not o.is_contiguous():
        raise ValueError("o must be a contiguous bfloat16 CUDA tensor [B, H, N, D]")
    B, H, N, D = o.shape
    if w_o.dim() != 2 or w_o.shape[1] != H * D or w_o.dtype != torch.bfloat16 or not w_o.is_contiguous():
        raise ValueError("w_o must be a contiguous bfloat16 [C_out, H*D] tensor")
    C_out = w_o.shape[0]
    y = _empty(stream, torch.bfloat16, o.device, B, N, C_out) if y is None else y
    ws = ws if ws is not None else _proj_workspace(o.device, stream)
    _check(load().sv_out_projection(_ptr(o), _ptr(w_o), _ptr(y), B, N, H, D, C_out, ws.ptr, ws.nbytes, _stream(stream)))
    return y


def rope_pairs(D: int):
    """A split of the D/2 rotation pairs over (frame, row, column): row and column get D // 6 pairs
    each, the frame axis the rest (22, 21, 21 for D = 128)."""
    ph = D // 6
    return (D // 2 - 2 * ph, ph, ph)


def sv_rope3d_table_bytes(frames: int, height: int, width: int, D: int) -> int:
    n = load().sv_rope3d_table_bytes(frames, height, width, D)
    if n == 0:
        raise SvError(SV_ERR_INVALID_ARG, load().sv_last_error().decode())
    return n


class Rope3dTable:
    """The device (cos, sin) table of the 3D rotary embedding for one grid and feature split, built
    by sv_rope3d_table; `desc(frame0)` gives the sv_rope3d descriptor of a call."""

    def __init__(self, frames: int, height: int, width: int, D: int, pairs, base: float = 10000.0, device=None,
                 stream=None):
        pt, ph, pw = (int(p) for p in pairs)
        nbytes = sv_rope3d_table_bytes(frames, height, width, D)
        self.table = _empty(stream, torch.float32, device or torch.device("cuda"), nbytes // 4)
        self.frames, self.height, self.width, self.D, self.pairs = frames, height, width, D, (pt, ph, pw)
        _check(load().sv_rope3d_table(self.table.data_ptr(), nbytes, frames, height, width, D, pt, ph, pw, base,
                                      _stream(stream)))

    def desc(self, frame0: int = 0) -> SvRope3d:
        pt, ph, pw = self.pairs
        return SvRope3d(self.table.data_ptr(), self.frames, self.height, self.width, self.D, pt, ph, pw, int(frame0))


def sv_rope3d_table(frames: int, height: int, width: int, D: int, pairs, base: float = 10000.0, device=None,
                    stream=None) -> Rope3dTable:
    return Rope3dTable(frames, height, width, D, pairs, base, device, stream)


def sv_block_causal_attn_rope(q, k, v, block_len: int, rope: Rope3dTable, frame0: int = 0, o=None, eps: float = 1e-6,
                              S_in=None, z_in=None, S_out=None, z_out=None, ws: Workspace | None = None, stream=None):
    """sv_block_causal_attn with the 3D rotary embedding of the numerator; returns o."""
    o = _empty_like(q, stream) if o is None else o
    B, H, N, D = _qkv(q, k, v, o)
    for t in (S_in, z_in, S_out, z_out):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or t.device != q.device):
            raise ValueError("S/z must be contiguous float32 tensors on q's device")
    if rope.table.device != q.device:
        raise ValueError("the rope table must live on q's device")
    ws = _ws(ws, SV_OP_BLOCK_CAUSAL_ATTN, q, block_len, stream)
    d = rope.desc(frame0)
    _check(load().sv_block_causal_attn_rope(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, D, int(block_len), _dt(q),
                                            eps, _ptr(S_in), _ptr(z_in), _ptr(S_out), _ptr(z_out), ctypes.byref(d),
                                            ws.ptr, ws.nbytes, _stream(stream)))
    return o


_MX_BLOCK = (32, 32, 16)     # by format: columns in a block
_MX_RUN = (128, 256, 256)    # columns in 128 bytes of codes


def _mx_scale_shape(rows, cols, fmt):
    run = _MX_RUN[fmt]
    return (-(-rows // 128), -(-cols // run) * (run // _MX_BLOCK[fmt]) // 4, 32, 4, 4)


def _mx_sizes(rows, cols, fmt):
    """(bytes of codes rounded up to 256, bytes of scales)."""
    run = _MX_RUN[fmt]
    return ((rows * cols if fmt == SV_MXFP8 else rows * cols // 2) + 255 & -256,
            (rows + 127 & -128) * (-(-cols // run) * (run // _MX_BLOCK[fmt])))


class MxTensor:
    """A microscaled matrix [rows, cols] (formats and layout: include/svlinattn.h).

    codes: uint8 [rows, cols] (SV_MXFP8) or [rows, cols / 2]; scales: uint8 [row tiles, block tiles, 32, 4, 4];
    gscale: float32 [1], the tensor scale of SV_NVFP4, None for the other formats. The tensors are read
    at every call: change them in place, or make another MxTensor (the fields cannot be assigned).
    """

    __slots__ = ("_codes", "_scales", "_buf", "_gscale", "_rows", "_cols", "_fmt", "_device", "_c", "_ref")

    def __init__(self, codes, scales, rows: int, cols: int, fmt: int, gscale=None):
        _mx_check(rows, cols, fmt, gscale, codes.device)
        if not codes.is_cuda:
            raise ValueError("codes must live on a CUDA device")
        if codes.dtype != torch.uint8 or codes.shape != (rows, cols if fmt == SV_MXFP8 else cols // 2) or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous uint8 tensor [rows, cols] (SV_MXFP8) or [rows, cols / 2]")
        if (scales.dtype != torch.uint8 or scales.shape != _mx_scale_shape(rows, cols, fmt) or not scales.is_contiguous()
                or scales.device != codes.device):
            raise ValueError(f"scales must be a contiguous uint8 tensor {_mx_scale_shape(rows, cols, fmt)} on codes' device")
        self._codes, self._scales, self._buf = codes, scales, None
        self._rows, self._cols, self._fmt, self._gscale, self._device = rows, cols, fmt, gscale, codes.device
        self._c = SvMx(codes.data_ptr(), scales.data_ptr(), None if gscale is None else gscale.data_ptr(), rows, cols, fmt)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, rows: int, cols: int, fmt: int, gscale=None, device=None):
        """An MxTensor with uninitialised codes and scales (an output for sv_mx_quantize or sv_rmsnorm)."""
        if device is None:
            device = gscale.device if gscale is not None else torch.device("cuda", torch.cuda.current_device())
        else:
            device = torch.device(device)
            if device.type == "cuda" and device.index is None:
                device = torch.device("cuda", torch.cuda.current_device())
        return cls._new(rows, cols, fmt, gscale, device)

    @classmethod
    def _new(cls, rows, cols, fmt, gscale, device, stream=None):
        _mx_check(rows, cols, fmt, gscale, device)
        m = cls.__new__(cls)
        n, ns = _mx_sizes(rows, cols, fmt)  # one allocation; codes and scales are views made when asked for
        m._buf = buf = (torch.empty(n + ns, dtype=torch.uint8, device=device) if stream is None
                        else _empty(stream, torch.uint8, device, n + ns))
        m._codes = m._scales = None
        m._rows, m._cols, m._fmt, m._gscale, m._device = rows, cols, fmt, gscale, buf.device
        p = buf.data_ptr()
        m._c = c = SvMx(p, p + n, None if gscale is None else gscale.data_ptr(), rows, cols, fmt)
        m._ref = ctypes.byref(c)
        return m

    # read-only: the descriptor that the calls take holds what they were when it was made
    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    fmt = property(lambda self: self._fmt)
    gscale = property(lambda self: self._gscale)
    device = property(lambda self: self._device)

    @property
    def codes(self):
        if self._codes is None:
            c = self._cols if self._fmt == SV_MXFP8 else self._cols // 2
            self._codes = self._buf.as_strided((self._rows, c), (c, 1), 0)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            shape = _mx_scale_shape(self._rows, self._cols, self._fmt)
            n = _mx_sizes(self._rows, self._cols, self._fmt)[0]
            self._scales = self._buf.as_strided(shape, (shape[1] * 512, 512, 16, 4, 1), n)
        return self._scales


def _mx_check(rows, cols, fmt, gscale, device):
    if fmt not in (SV_MXFP8, SV_MXFP4, SV_NVFP4):
        raise ValueError("fmt must be SV_MXFP8, SV_MXFP4 or SV_NVFP4")
    if rows < 1 or not 32 <= cols < 1 << 31 or cols % 32 != 0:  # cols goes to the library as an int
        raise ValueError("rows must be >= 1 and cols a positive multiple of 32 below 2^31")
    if gscale is None:
        if fmt == SV_NVFP4:
            raise ValueError("SV_NVFP4 needs a tensor scale gscale")
    elif fmt != SV_NVFP4:
        raise ValueError("only SV_NVFP4 takes a tensor scale")
    elif (gscale.dtype != torch.float32 or gscale.numel() != 1 or gscale.device != device):
        raise ValueError("gscale must be a float32 tensor of one value on codes' device")


def _call(fn, index, args):
    """fn(*args) with device `index` current (tensors may live on another device than the current one);
    raises on an error."""
    if index == _current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(index):
            st = fn(*args)
    if st != SV_OK:
        _check(st)


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_current_device = torch.cuda.current_device
if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same handle without a Stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream
if hasattr(torch._C, "_cuda_getDevice"):  # the same index; there is a CUDA tensor, so CUDA is initialised
    _current_device = torch._C._cuda_getDevice


def _mx_out(out, rows, cols, fmt, gscale, device, stream):
    if out is None:
        return MxTensor._new(rows, cols, fmt, gscale, device, stream)
    if out._rows != rows or out._cols != cols or out._fmt != fmt or out._device != device:
        raise ValueError(f"out must be a microscaled [{rows}, {cols}] matrix of the call's format on x's device")
    if gscale is not None and gscale is not out._gscale:
        raise ValueError("gscale must be out's own tensor scale, or None")
    return out


def _dense(x):
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor")


def sv_mx_global_scale(x, g=None, stream=None):
    """The tensor scale of SV_NVFP4: max |x| / (6 * 448) as a float32 tensor [1] (g, when given)."""
    _dense(x)
    device = x.device
    index = device.index
    if g is None:
        g = _empty(stream, torch.float32, device, 1)
    elif g.dtype != torch.float32 or g.numel() != 1 or g.device != device:
        raise ValueError("g must be a float32 tensor of one value on x's device")
    _call(load().sv_mx_global_scale, index, (x.data_ptr(), x.numel(), _dt(x), g.data_ptr(),
                                             _raw_stream(index) if stream is None else stream.cuda_stream))
    return g


def sv_mx_quantize(x, fmt: int, gscale=None, out: MxTensor | None = None, stream=None) -> MxTensor:
    """x to a microscaled matrix: [..., C] rows as they are, or [B, H, N, D] (four dimensions) as B * N
    rows that hold the heads side by side. SV_NVFP4 takes the tensor scale gscale (float32 [1])."""
    _dense(x)
    shape, device = x.shape, x.device
    index = device.index
    if len(shape) == 4:
        B, H, N, D = shape
    elif len(shape) >= 2:
        B, H, D = 1, 1, shape[-1]
        N = x.numel() // D if D else 0
    else:
        raise ValueError("x must be [..., C] or [B, H, N, D]")
    out = _mx_out(out, B * N, H * D, fmt, gscale, device, stream)
    _call(load().sv_mx_quantize, index, (x.data_ptr(), B, H, N, D, _dt(x), out._ref,
                                         _raw_stream(index) if stream is None else stream.cuda_stream))
    return out


def sv_mx_dequantize(xq: MxTensor, dtype=torch.bfloat16, y=None, stream=None):
    """The values of a microscaled matrix as [rows, cols] bfloat16 or float32."""
    index = xq._device.index
    if y is None:
        y = _empty(stream, dtype, xq._device, xq._rows, xq._cols)
    elif tuple(y.shape) != (xq._rows, xq._cols) or not y.is_contiguous() or y.device != xq._device:
        raise ValueError("y must be a contiguous [rows, cols] tensor on xq's device")
    _call(load().sv_mx_dequantize, index, (xq._ref, y.data_ptr(), _dt(y),
                                           _raw_stream(index) if stream is None else stream.cuda_stream))
    return y


def sv_rmsnorm(x, w, residual=None, eps: float = 1e-6, fmt: int | None = None, gscale=None, h=None, y=None, stream=None):
    """Root-mean-square norm over x's last dimension after the residual's addition; returns (y, h).

    h = x + residual in x's dtype (x itself without a residual; None where y overwrites it, that is, without a
    residual and with y in x's place). y = h / rms(h) * w, in x's dtype and shape,
    or, with fmt, quantised in the same pass to an MxTensor of one row per position (y, when given, is that
    MxTensor; SV_NVFP4 takes gscale). h may be x or residual (in place)."""
    _dense(x)
    shape, dtype, device = x.shape, x.dtype, x.device
    index = device.index
    C = shape[-1] if len(shape) else 0
    rows = x.numel() // C if C else 0
    if rows == 0 or C > 32768:  # C goes to the library as an int
        raise ValueError("x must be [..., C] with at least one row and column, and C at most 32768")
    if w.dtype != torch.float32 or w.shape != (C,) or not w.is_contiguous() or w.device != device:
        raise ValueError("w must be a contiguous float32 [C] tensor on x's device")
    if residual is None:
        if h is not None and h is not x:
            raise ValueError("without a residual h is x")
        h = x
        pr = ph = None
    else:
        for t in (residual,) if h is None else (residual, h):
            if t is not x and (t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous()):
                raise ValueError("residual and h must be contiguous tensors of x's shape, dtype and device")
        if h is None:
            h = torch.empty_like(x) if stream is None else _empty_like(x, stream)
        pr, ph = residual.data_ptr(), h.data_ptr()
    if fmt is None:
        if gscale is not None:
            raise ValueError("gscale goes with fmt=SV_NVFP4")
        if y is None:
            y = _empty_like(x, stream)
        elif y.shape != shape or y.dtype != dtype or y.device != device or not y.is_contiguous():
            raise ValueError("y must be a contiguous tensor of x's shape, dtype and device")
        py, pq = y.data_ptr(), None
        if residual is None and py == x.data_ptr():
            h = None  # the sum is overwritten
    else:
        y = _mx_out(y, rows, C, fmt, gscale, device, stream)
        py, pq = None, y._ref
    _call(load().sv_rmsnorm, index, (x.data_ptr(), pr, ph, w.data_ptr(), rows, C, _dt(x), eps, py, pq,
                                     _raw_stream(index) if stream is None else stream.cuda_stream))
    return y, h


_mx_ws = {}  # (device index, stream handle): the products' workspace; device index: that of captured calls
_mx_ws_lock = threading.Lock()


def _capturing(stream):
    if torch.cuda.is_current_stream_capturing():
        return True
    if stream is None:
        return False
    with _on(stream):
        return torch.cuda.is_current_stream_capturing()


def _mx_workspace(ws, device, handle, stream):
    """The caller's workspace, else one kept per (device, stream), so that a timeout is reported to the stream
    whose call ran into it. Calls captured on a stream without one share the device's workspace for captures (they
    use its status word only, and a raised word stops no product); no call sees their replays, so the
    device's next call reports for them. Raises if an earlier call on the workspace timed out."""
    if ws is not None:
        if ws.buf.device != device:
            raise ValueError("ws must be a workspace on x's device")
        ws.check(stream)
        return ws
    index = device.index
    ws = _mx_ws.get((index, handle))
    if ws is None:
        ws = _mx_make_workspace(device, handle, stream)
    captured = _mx_ws[index]
    if captured._word[0]:
        captured.check(stream)
    if ws._word[0]:
        ws.check(stream)
    return ws


def _mx_make_workspace(device, handle, stream):
    index = device.index
    if _capturing(stream):
        ws = _mx_ws.get(index)
        if ws is None:
            raise RuntimeError("the microscaled products' workspace must exist before a capture: make a call first, or pass ws")
        return ws
    with _mx_ws_lock, torch.cuda.device(device):
        for key in (index, (index, handle)):
            if key not in _mx_ws:
                _mx_ws[key] = Workspace(256, device, stream)
        return _mx_ws[index, handle]


def _mx_pair(xq, wq):
    if xq._fmt != wq._fmt or xq._cols != wq._cols or xq._device != wq._device:
        raise ValueError("x and w must share format, number of columns and device")


def sv_mx_projection(xq: MxTensor, wq: MxTensor, y=None, ws: Workspace | None = None, stream=None):
    """y [xq.rows, wq.rows] bfloat16 = x W^T of two microscaled matrices. Make the first call on a device
    (or pass ws) before capturing one into a CUDA graph."""
    _mx_pair(xq, wq)
    device = xq._device
    index = device.index
    if y is None:
        y = (torch.empty(xq._rows, wq._rows, dtype=torch.bfloat16, device=device) if stream is None
             else _empty(stream, torch.bfloat16, device, xq._rows, wq._rows))
    elif (y.dtype != torch.bfloat16 or y.numel() != xq._rows * wq._rows or y.shape[-1] != wq._rows or not y.is_contiguous()
            or y.device != device):
        raise ValueError("y must be a contiguous bfloat16 tensor of x's rows and w's rows on x's device")
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    ws = _mx_workspace(ws, device, handle, stream)
    _call(load().sv_mx_projection, index, (xq._ref, wq._ref, y.data_ptr(), ws.ptr, ws.nbytes, handle))
    return y


def sv_mx_qkv_projection(xq: MxTensor, wq: MxTensor, B: int, N: int, H: int, D: int, q=None, k=None, v=None,
                         ws: Workspace | None = None, stream=None):
    """x of B * N rows, w of 3 * H * D rows -> (ReLU(q), ReLU(k), v), each [B, H, N, D] bfloat16. ws as for
    sv_mx_projection."""
    _mx_pair(xq, wq)
    device = xq._device
    index = device.index
    if B * N != xq._rows or 3 * H * D != wq._rows:
        raise ValueError("x must have B * N rows and w 3 * H * D rows")
    for t in (q, k, v):
        if t is not None and (t.shape != (B, H, N, D) or t.dtype != torch.bfloat16 or not t.is_contiguous()
                              or t.device != device):
            raise ValueError("q, k, v must be contiguous bfloat16 [B, H, N, D] tensors on x's device")
    q, k, v = (_empty(stream, torch.bfloat16, device, B, H, N, D) if t is None else t
               for t in (q, k, v))
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    ws = _mx_workspace(ws, device, handle, stream)
    _call(load().sv_mx_qkv_projection, index, (xq._ref, wq._ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), B, N, H, D,
                                               ws.ptr, ws.nbytes, handle))
    return q, k, v
