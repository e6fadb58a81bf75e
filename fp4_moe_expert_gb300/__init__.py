"""Python binding of libfme.so (include/fme.h): the routed-expert MoE decode
layer (FP8 and NVFP4) and the FP8 shared expert on sm_103a.

Argument marshalling only: torch supplies device memory and the current
stream; every step of the computation runs in the library's CUDA kernels.
Importing this package loads libfme.so and raises if it is missing (build it
with ``python -m fp4_moe_expert_gb300.build`` or ``__graft_entry__.build()``).
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfme.so")

FME_OK = 0
FME_F32 = 0
FME_BF16 = 1

# Every symbol include/fme.h declares, with its ctypes signature.
_c_int, _c_size, _vp, _c_float = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
_c_ll = ctypes.c_longlong
SIGNATURES = {
    "fme_last_error": (ctypes.c_char_p, []),
    "fme_version": (_c_int, []),
    "fme_moe_routed_fp8": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                    _c_int, _c_float, _c_float, _c_int, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "fme_moe_routed_fp8_workspace": (_c_size, [_c_int] * 5),
    "fme_moe_routed_fp8_mx": (_c_int, [_vp, _vp, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                       _c_int, _c_float, _c_float, _c_int, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "fme_moe_routed_fp8_noalloc": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                            _c_int, _c_int, _c_float, _c_float, _c_int, _vp, _vp, _vp, _vp]),
    "fme_moe_routed_fp8_noalloc_error": (_c_int, [_vp, _vp]),
    "fme_shared_expert_fp8": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_float, _c_int, _vp,
                                       _vp, _vp, _c_size, _vp]),
    "fme_shared_expert_fp8_workspace": (_c_size, [_c_int] * 3),
    "fme_moe_layer_fp8": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                   _c_int, _c_float, _c_float, _c_int, _vp, _vp, _vp, _vp, _c_float, _c_int,
                                   _vp, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "fme_moe_layer_fp8_workspace": (_c_size, [_c_int] * 5),
    "fme_ue8m0_unpack": (_c_int, [_vp, _c_int, _c_int, _vp, _c_int, _vp, _vp]),
    "fme_moe_routed_nvfp4": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                      _c_int, _c_float, _vp, _vp, _c_size, _vp]),
    "fme_moe_routed_nvfp4_workspace": (_c_size, [_c_int] * 5),
    "fme_moe_finalize": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp]),
    "fme_mxfp8_quantize": (_c_int, [_vp, _c_int, _c_int, _vp, _vp, _vp]),
    "fme_combine_rmsnorm": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _c_float, _vp, _vp, _vp]),
    "fme_moe_layer_nvfp4": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                     _c_int, _c_int, _c_int, _c_float, _c_float, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "fme_add_rmsnorm_fp8": (_c_int, [_vp, _c_ll, _vp, _c_ll, _vp, _c_int, _c_int, _c_float, _c_int, _vp, _vp, _vp,
                                     _vp, _vp]),
    "fme_add_rmsnorm_mxfp8": (_c_int, [_vp, _c_ll, _vp, _c_ll, _vp, _c_int, _c_int, _c_float, _vp, _vp, _vp, _vp,
                                       _vp]),
    "fme_moe_route": (_c_int, [_vp, _c_int, _vp, _c_int, _c_int, _c_int, _c_float, _vp, _vp, _vp, _vp, _vp, _vp,
                               _c_size, _vp]),
    "fme_moe_route_workspace": (_c_size, [_c_int] * 3),
    "fme_moe_grouped_swiglu_fp8": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                            _c_float, _c_int, _c_int, _vp, _vp, _vp, _c_size, _vp]),
    "fme_moe_grouped_gemm_fp8": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                          _vp, _c_int, _vp, _c_size, _vp]),
    "fme_moe_grouped_fp8_workspace": (_c_size, [_c_int] * 4),
    "fme_workspace_clear": (_c_int, [_vp, _c_size, _vp]),
    "fme_selftest_wait_timeout": (_c_int, [_vp, _c_size, _c_int, _vp]),
    "fme_selftest_rounding": (_c_int, [_c_int, ctypes.c_uint32, ctypes.c_ulonglong, _vp, _vp]),
    "fme_workspace_error": (_c_int, [_vp, ctypes.POINTER(_c_int), _vp]),
    "fme_sm_count": (_c_int, []),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libfme.so not built at {LIB_PATH}; run fp4_moe_expert_gb300/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class FmeError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"fme status {status}: {message}")
        self.status = status


def _check(status):
    if status != FME_OK:
        raise FmeError(status, lib.fme_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without a Stream object (2 us less a call); the public route where it is missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need(t, dtype, shape, name, device=None):
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, the other operands on {device}")
    if t.dtype != dtype or t.shape != torch.Size(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)} contiguous={t.is_contiguous()} cuda={t.is_cuda}")


class Workspace:
    """Caller-owned device scratch for one stream: zero-filled once at creation;
    every successful call leaves it zeroed again."""

    def __init__(self, nbytes, device):
        self.nbytes = int(nbytes)
        self.buf = torch.zeros(max(self.nbytes, 256), dtype=torch.uint8, device=device)

    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    def clear(self):
        _check(lib.fme_workspace_clear(self.ptr(), self.nbytes, _stream(self.buf.device)))

    def error(self):
        """Device error word (0 = none); reading it synchronises the stream and clears it."""
        code = ctypes.c_int(0)
        lib.fme_workspace_error(self.ptr(), ctypes.byref(code), _stream(self.buf.device))
        return code.value


_ws_cache = {}


def _workspace(nbytes, device, workspace):
    if workspace is not None:
        if workspace.nbytes < nbytes:
            raise ValueError(f"workspace of {workspace.nbytes} bytes, {nbytes} needed")
        return workspace
    key = (device.index if device.index is not None else torch.cuda.current_device(), nbytes)
    ws = _ws_cache.get(key)
    if ws is None:
        ws = Workspace(nbytes, device)
        _ws_cache[key] = ws
    return ws


def kept_workspace_error(device=None):
    """Device error bits (Workspace.error, or-ed; 0 = none) of the workspaces kept for calls that were given none, on
    `device` (default: the current one). Synchronises the device. A workspace with an error is cleared, so that later
    calls are right again; what the calls since the error returned is not."""
    index = None if device is None else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    torch.cuda.synchronize(index)
    bits = 0
    for key, ws in list(_ws_cache.items()):
        if key[0] == index:
            code = ws.error()
            if code != 0:
                ws.clear()
            bits |= code
    torch.cuda.synchronize(index)
    return bits


def moe_routed_fp8_workspace(M, H, I, E, top_k):
    return lib.fme_moe_routed_fp8_workspace(M, H, I, E, top_k)


def moe_routed_fp8(x, logits, bias, w13, s13, w2, s2, top_k, limit, scale, ue8m0,
                   out=None, ids=None, weights=None, workspace=None):
    """Routed FP8 experts of M tokens (fme_moe_routed_fp8).

    x [M, H] bf16; logits [M, E] bf16 or float32; bias [E] float32;
    w13 [E, 2I, H] uint8 (E4M3, up rows then gate rows); s13 [E, 2I/128, H/128] f32;
    w2 [E, H, I] uint8; s2 [E, H/128, I/128] f32.
    Returns out [M*top_k, H] bf16 (unweighted route rows), ids [M, top_k] int32,
    weights [M, top_k] float32.
    """
    M, H = x.shape
    E, n2, _ = w13.shape
    I = n2 // 2
    dev = x.device
    _need(x, torch.bfloat16, (M, H), "x")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be float32 or bfloat16")
    _need(logits, logits.dtype, (M, E), "logits")
    _need(bias, torch.float32, (E,), "bias")
    _need(w13, torch.uint8, (E, 2 * I, H), "w13")
    _need(s13, torch.float32, (E, 2 * I // 128, H // 128), "s13")
    _need(w2, torch.uint8, (E, H, I), "w2")
    _need(s2, torch.float32, (E, H // 128, I // 128), "s2")
    if out is None:
        out = torch.empty(M * top_k, H, dtype=torch.bfloat16, device=dev)
    if ids is None:
        ids = torch.empty(M, top_k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(M, top_k, dtype=torch.float32, device=dev)
    need = moe_routed_fp8_workspace(M, H, I, E, top_k)
    ws = _workspace(need, dev, workspace)
    ldt = FME_F32 if logits.dtype == torch.float32 else FME_BF16
    _check(lib.fme_moe_routed_fp8(_ptr(x), _ptr(logits), ldt, _ptr(bias), _ptr(w13), _ptr(s13), _ptr(w2),
                                  _ptr(s2), M, H, I, E, top_k, float(limit), float(scale), int(bool(ue8m0)),
                                  _ptr(out), _ptr(ids), _ptr(weights), ws.ptr(), ws.nbytes, _stream(dev)))
    return out, ids, weights


def moe_routed_fp8_mx(xq, xscales, logits, bias, w13, s13, w2, s2, top_k, limit, scale, ue8m0,
                      out=None, ids=None, weights=None, workspace=None):
    """moe_routed_fp8 with MXFP8 activations (fme_moe_routed_fp8_mx): xq [M, H] uint8
    E4M3 and xscales [M, H/32] uint8 E8M0 (as mxfp8_quantize returns). Returns
    (out [M*top_k, H] bf16, ids [M, top_k] int32, weights [M, top_k] float32)."""
    M, H = xq.shape
    E = logits.shape[1]
    I = w2.shape[2]
    dev = xq.device
    _need(xq, torch.uint8, (M, H), "xq")
    _need(xscales, torch.uint8, (M, H // 32), "xscales")
    if logits.dtype == torch.float32:
        dt = FME_F32
    elif logits.dtype == torch.bfloat16:
        dt = FME_BF16
    else:
        raise ValueError("logits must be float32 or bfloat16")
    _need(logits, logits.dtype, (M, E), "logits")
    _need(bias, torch.float32, (E,), "bias")
    _need(w13, torch.uint8, (E, 2 * I, H), "w13")
    _need(s13, torch.float32, (E, 2 * I // 128, H // 128), "s13")
    _need(w2, torch.uint8, (E, H, I), "w2")
    _need(s2, torch.float32, (E, H // 128, I // 128), "s2")
    if out is None:
        out = torch.empty(M * top_k, H, dtype=torch.bfloat16, device=dev)
    if ids is None:
        ids = torch.empty(M, top_k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(M, top_k, dtype=torch.float32, device=dev)
    need = moe_routed_fp8_workspace(M, H, I, E, top_k)
    ws = _workspace(need, dev, workspace)
    _check(lib.fme_moe_routed_fp8_mx(_ptr(xq), _ptr(xscales), _ptr(logits), dt, _ptr(bias), _ptr(w13), _ptr(s13),
                                     _ptr(w2), _ptr(s2), M, H, I, E, top_k, float(limit), float(scale), int(ue8m0),
                                     _ptr(out), _ptr(ids), _ptr(weights), ws.ptr(), ws.nbytes, _stream(dev)))
    return out, ids, weights


def shared_expert_fp8_workspace(M, H, I):
    return lib.fme_shared_expert_fp8_workspace(M, H, I)


def shared_expert_fp8(x, w13, s13, w2, s2, limit, ue8m0, out=None, gate_up=None, want_gate_up=False,
                      workspace=None):
    """FP8 shared expert (fme_shared_expert_fp8). w13 [2I, H] (gate rows first),
    s13 [2I/128, H/128] f32, w2 [H, I], s2 [H/128, I/128] f32. Returns out [M, H]
    bf16 (and gate_up [M, 2I] bf16 when want_gate_up)."""
    M, H = x.shape
    n2 = w13.shape[0]
    I = n2 // 2
    dev = x.device
    _need(x, torch.bfloat16, (M, H), "x")
    _need(w13, torch.uint8, (2 * I, H), "w13")
    _need(s13, torch.float32, (2 * I // 128, H // 128), "s13")
    _need(w2, torch.uint8, (H, I), "w2")
    _need(s2, torch.float32, (H // 128, I // 128), "s2")
    if out is None:
        out = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    if want_gate_up and gate_up is None:
        gate_up = torch.empty(M, 2 * I, dtype=torch.bfloat16, device=dev)
    need = shared_expert_fp8_workspace(M, H, I)
    ws = _workspace(need, dev, workspace)
    _check(lib.fme_shared_expert_fp8(_ptr(x), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), M, H, I, float(limit),
                                     int(bool(ue8m0)), _ptr(gate_up), _ptr(out), ws.ptr(), ws.nbytes,
                                     _stream(dev)))
    return (out, gate_up) if want_gate_up else out


def moe_layer_fp8_workspace(M, H, I, E, top_k):
    return lib.fme_moe_layer_fp8_workspace(M, H, I, E, top_k)


def moe_layer_fp8(x, logits, bias, w13, s13, w2, s2, top_k, limit, scale, ue8m0,
                  shared_w13, shared_s13, shared_w2, shared_s2, shared_limit, shared_ue8m0,
                  out=None, ids=None, weights=None, shared_out=None, workspace=None):
    """Routed experts and shared expert in one launch (fme_moe_layer_fp8).

    Routed arguments as moe_routed_fp8; shared_* as shared_expert_fp8 (same H, I).
    Returns (out [M*top_k, H], ids, weights, shared_out [M, H]).
    """
    M, H = x.shape
    E, n2, _ = w13.shape
    I = n2 // 2
    dev = x.device
    _need(x, torch.bfloat16, (M, H), "x")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be float32 or bfloat16")
    _need(logits, logits.dtype, (M, E), "logits")
    _need(bias, torch.float32, (E,), "bias")
    _need(w13, torch.uint8, (E, 2 * I, H), "w13")
    _need(s13, torch.float32, (E, 2 * I // 128, H // 128), "s13")
    _need(w2, torch.uint8, (E, H, I), "w2")
    _need(s2, torch.float32, (E, H // 128, I // 128), "s2")
    _need(shared_w13, torch.uint8, (2 * I, H), "shared_w13")
    _need(shared_s13, torch.float32, (2 * I // 128, H // 128), "shared_s13")
    _need(shared_w2, torch.uint8, (H, I), "shared_w2")
    _need(shared_s2, torch.float32, (H // 128, I // 128), "shared_s2")
    if out is None:
        out = torch.empty(M * top_k, H, dtype=torch.bfloat16, device=dev)
    if ids is None:
        ids = torch.empty(M, top_k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(M, top_k, dtype=torch.float32, device=dev)
    if shared_out is None:
        shared_out = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    need = moe_layer_fp8_workspace(M, H, I, E, top_k)
    ws = _workspace(need, dev, workspace)
    ldt = FME_F32 if logits.dtype == torch.float32 else FME_BF16
    _check(lib.fme_moe_layer_fp8(_ptr(x), _ptr(logits), ldt, _ptr(bias), _ptr(w13), _ptr(s13), _ptr(w2),
                                 _ptr(s2), M, H, I, E, top_k, float(limit), float(scale), int(bool(ue8m0)),
                                 _ptr(shared_w13), _ptr(shared_s13), _ptr(shared_w2), _ptr(shared_s2),
                                 float(shared_limit), int(bool(shared_ue8m0)), _ptr(out), _ptr(ids),
                                 _ptr(weights), _ptr(shared_out), ws.ptr(), ws.nbytes, _stream(dev)))
    return out, ids, weights, shared_out


def moe_finalize(out, weights, shared_out=None, y=None):
    """y [M, H] BF16 = bf16(sum over r of weights[t, r] * out[t * top_k + r] (+ shared_out[t]))
    (fme_moe_finalize): out [M * top_k, H] BF16 unweighted expert rows as the routed
    call returns them, weights [M, top_k] FP32, shared_out [M, H] BF16 or None."""
    dev = out.device
    M, top_k = weights.shape
    H = out.shape[1]
    _need(out, torch.bfloat16, (M * top_k, H), "out")
    _need(weights, torch.float32, (M, top_k), "weights")
    if shared_out is not None:
        _need(shared_out, torch.bfloat16, (M, H), "shared_out")
    if y is None:
        y = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    _need(y, torch.bfloat16, (M, H), "y")
    _check(lib.fme_moe_finalize(_ptr(out), _ptr(weights), _ptr(shared_out), M, H, top_k, _ptr(y), _stream(dev)))
    return y


def mxfp8_quantize(x):
    """(q [T, H] uint8 E4M3, scales [T, H/32] uint8 E8M0) of x [T, H] BF16 (fme_mxfp8_quantize)."""
    T, H = x.shape
    dev = x.device
    _need(x, torch.bfloat16, (T, H), "x")
    q = torch.empty(T, H, dtype=torch.uint8, device=dev)
    sc = torch.empty(T, H // 32, dtype=torch.uint8, device=dev)
    _check(lib.fme_mxfp8_quantize(_ptr(x), T, H, _ptr(q), _ptr(sc), _stream(dev)))
    return q, sc


def combine_rmsnorm(partials, gamma, eps=1e-5):
    """(latent [T, H], normed [T, H]) BF16 of partials [T, N, H] BF16 and gamma [H] BF16
    (fme_combine_rmsnorm)."""
    T, N, H = partials.shape
    dev = partials.device
    _need(partials, torch.bfloat16, (T, N, H), "partials")
    _need(gamma, torch.bfloat16, (H,), "gamma")
    latent = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    normed = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    _check(lib.fme_combine_rmsnorm(_ptr(partials), T, N, H, _ptr(gamma), float(eps), _ptr(latent), _ptr(normed),
                                   _stream(dev)))
    return latent, normed


def ue8m0_unpack(packed, n, k, check=True):
    """FP32 [n/128, k/128] block scales from packed UE8M0 int32 [n, k/512]
    (fme_ue8m0_unpack). With check, raises ValueError when a 128-row block is
    not uniform (this reads a device flag, so it synchronises)."""
    dev = packed.device
    _need(packed, torch.int32, (n, k // 512), "packed")
    dst = torch.empty(n // 128, k // 128, dtype=torch.float32, device=dev)
    flag = torch.zeros(4, dtype=torch.int32, device=dev) if check else None
    _check(lib.fme_ue8m0_unpack(_ptr(packed), n, k, _ptr(dst), int(check), _ptr(flag), _stream(dev)))
    if check and int(flag[0].item()) != 0:
        raise ValueError("scales vary inside a 128-row block")
    return dst


def _stream_workspace(nbytes, device, workspace):
    """The caller's workspace, or one kept per device, current stream and size. A graph capture gets a new one, the
    graph's own: zeroed in every replay, and shared neither with calls outside the graph nor with another graph."""
    if workspace is not None:
        if workspace.buf.device != device:
            raise ValueError(f"workspace: on {workspace.buf.device}, the operands on {device}")
        return _workspace(nbytes, device, workspace)
    if torch.cuda.is_current_stream_capturing():
        return Workspace(nbytes, device)
    key = (device.index, _stream(device), nbytes)
    ws = _ws_cache.get(key)
    if ws is None:
        ws = _ws_cache[key] = Workspace(nbytes, device)
    return ws


def _launch_stream(device):
    """The current stream of the operands' device, which has to be the current device: kernels launch there."""
    if device.index != torch.cuda.current_device():
        raise ValueError(f"operands on {device}, but the current device is cuda:{torch.cuda.current_device()}")
    return _stream(device)


def _rows(t, name):
    """Row stride of a BF16 CUDA matrix with contiguous rows."""
    if t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_cuda or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a CUDA bfloat16 matrix with contiguous rows, got {t.dtype} "
                         f"{tuple(t.shape)} strides={t.stride()} cuda={t.is_cuda}")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 8)


def _out(t, shape, dtype, device, name):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, dtype, shape, name, device)
    return t


def _addr(t):
    return None if t is None else t.data_ptr()


def _add_rmsnorm(x, gamma, residual, eps, mx, ue8m0, want_normed, q, scales, normed, residual_out):
    ldx, dev = _rows(x, "x"), x.device
    T, H = x.shape
    _need(gamma, torch.bfloat16, (H,), "gamma", dev)
    ldr = H
    if residual is not None:
        ldr = _rows(residual, "residual")
        if residual.shape != x.shape:
            raise ValueError(f"residual: expected {tuple(x.shape)}, got {tuple(residual.shape)}")
        if residual.device != dev:
            raise ValueError(f"residual: on {residual.device}, the other operands on {dev}")
        residual_out = _out(residual_out, (T, H), torch.bfloat16, dev, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    q = _out(q, (T, H), torch.uint8, dev, "q")
    scales = _out(scales, (T, H // (32 if mx else 128)), torch.uint8 if mx else torch.float32, dev, "scales")
    if want_normed or normed is not None:
        normed = _out(normed, (T, H), torch.bfloat16, dev, "normed")
    if T == 0:
        return q, scales, residual_out, normed
    if mx:
        st = lib.fme_add_rmsnorm_mxfp8(x.data_ptr(), ldx, _addr(residual), ldr, gamma.data_ptr(), T, H, eps,
                                       q.data_ptr(), scales.data_ptr(), _addr(normed), _addr(residual_out),
                                       _launch_stream(dev))
    else:
        st = lib.fme_add_rmsnorm_fp8(x.data_ptr(), ldx, _addr(residual), ldr, gamma.data_ptr(), T, H, eps,
                                     int(bool(ue8m0)), q.data_ptr(), scales.data_ptr(), _addr(normed),
                                     _addr(residual_out), _launch_stream(dev))
    _check(st)
    return q, scales, residual_out, normed


def add_rmsnorm_fp8(x, gamma, residual=None, eps=1e-5, ue8m0=False, want_normed=False, q=None, scales=None,
                    normed=None, residual_out=None):
    """Residual addition, RMSNorm and FP8 quantisation (fme_add_rmsnorm_fp8) of x [T, H] BF16 (any row stride) with
    gamma [H] BF16. Returns (q [T, H] uint8 E4M3, scales [T, H/128] float32, residual_out [T, H] BF16 or None without
    a residual, normed [T, H] BF16 or None unless wanted). residual_out may be residual itself."""
    return _add_rmsnorm(x, gamma, residual, eps, False, ue8m0, want_normed, q, scales, normed, residual_out)


def add_rmsnorm_mxfp8(x, gamma, residual=None, eps=1e-5, want_normed=False, q=None, scales=None, normed=None,
                      residual_out=None):
    """add_rmsnorm_fp8 in the MXFP8 format (fme_add_rmsnorm_mxfp8): scales [T, H/32] uint8 E8M0, as
    moe_routed_fp8_mx takes them."""
    return _add_rmsnorm(x, gamma, residual, eps, True, False, want_normed, q, scales, normed, residual_out)


def moe_route_workspace(T, E, top_k):
    return lib.fme_moe_route_workspace(T, E, top_k)


def moe_route(logits, bias, top_k, scale=1.0, ids=None, weights=None, offsets=None, rows=None, tokens=None,
              workspace=None):
    """Routing of T tokens and their routes grouped by expert (fme_moe_route): logits [T, E] bf16 or float32, bias [E]
    float32. Returns ids [T, top_k] int32, weights [T, top_k] float32, offsets [E + 1] int32 (expert e holds places
    offsets[e] .. offsets[e + 1] - 1), rows [T * top_k] int32 (the route t * top_k + r at each place) and tokens
    [T * top_k] int32 (its token)."""
    T, E = logits.shape
    dev = logits.device
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be float32 or bfloat16")
    _need(logits, logits.dtype, (T, E), "logits")
    _need(bias, torch.float32, (E,), "bias", dev)
    ids = _out(ids, (T, top_k), torch.int32, dev, "ids")
    weights = _out(weights, (T, top_k), torch.float32, dev, "weights")
    offsets = _out(offsets, (E + 1,), torch.int32, dev, "offsets")
    rows = _out(rows, (T * top_k,), torch.int32, dev, "rows")
    tokens = _out(tokens, (T * top_k,), torch.int32, dev, "tokens")
    if T == 0:
        return ids, weights, offsets.zero_(), rows, tokens
    ws = _stream_workspace(moe_route_workspace(T, E, top_k), dev, workspace)
    ldt = FME_F32 if logits.dtype == torch.float32 else FME_BF16
    _check(lib.fme_moe_route(logits.data_ptr(), ldt, bias.data_ptr(), T, E, top_k, scale, ids.data_ptr(),
                             weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), tokens.data_ptr(),
                             ws.buf.data_ptr(), ws.nbytes, _launch_stream(dev)))
    return ids, weights, offsets, rows, tokens


def moe_grouped_fp8_workspace(R, K, N, E):
    return lib.fme_moe_grouped_fp8_workspace(R, K, N, E)


def _need_grouped(a, sa, w, sw, offsets, in_rows):
    """Checks the operands the grouped products share; returns (a_rows, K, E, N, R)."""
    E, N, K = w.shape
    a_rows = a.shape[0]
    _need(a, torch.uint8, (a_rows, K), "a")
    _need(sa, torch.float32, (a_rows, K // 128), "sa", a.device)
    _need(w, torch.uint8, (E, N, K), "w", a.device)
    _need(sw, torch.float32, (E, N // 128, K // 128), "sw", a.device)
    _need(offsets, torch.int32, (E + 1,), "offsets", a.device)
    R = a_rows
    if in_rows is not None:
        R = in_rows.numel()
        _need(in_rows, torch.int32, (R,), "in_rows", a.device)
    return a_rows, K, E, N, R


def moe_grouped_swiglu_fp8(a, sa, w13, s13, offsets, in_rows=None, limit=float("inf"), ue8m0=False, gate_first=False,
                           q=None, scales=None, workspace=None):
    """Gate/up product, SwiGLU and FP8 re-quantisation of rows grouped by expert (fme_moe_grouped_swiglu_fp8).

    a [a_rows, H] uint8 E4M3 and sa [a_rows, H/128] float32; w13 [E, 2I, H] uint8 (up rows then gate rows, or the
    other way with gate_first) and s13 [E, 2I/128, H/128] float32; offsets [E + 1] int32; in_rows [R] int32 (the row
    of a at each place; None: the place itself). Returns q [R, I] uint8 E4M3 and scales [R, I/128] float32, at the
    places; places no group holds are left as they are."""
    a_rows, H, E, two_i, R = _need_grouped(a, sa, w13, s13, offsets, in_rows)
    I = two_i // 2
    dev = a.device
    q = _out(q, (R, I), torch.uint8, dev, "q")
    scales = _out(scales, (R, I // 128), torch.float32, dev, "scales")
    if R == 0:
        return q, scales
    ws = _stream_workspace(moe_grouped_fp8_workspace(R, H, two_i, E), dev, workspace)
    _check(lib.fme_moe_grouped_swiglu_fp8(a.data_ptr(), sa.data_ptr(), a_rows, w13.data_ptr(), s13.data_ptr(),
                                          offsets.data_ptr(), _addr(in_rows), R, H, I, E, limit, int(bool(ue8m0)),
                                          int(bool(gate_first)), q.data_ptr(), scales.data_ptr(), ws.buf.data_ptr(),
                                          ws.nbytes, _launch_stream(dev)))
    return q, scales


def moe_grouped_gemm_fp8(a, sa, w, sw, offsets, in_rows=None, out_rows=None, out=None, workspace=None):
    """Product of rows grouped by expert, BF16 out (fme_moe_grouped_gemm_fp8): a [a_rows, K], w [E, N, K] and their
    scales as moe_grouped_swiglu_fp8; out_rows [R] int32 (the output row of each place; None: the place itself).
    Returns out [R, N] BF16 (or the given out [out_n, N]); rows no place names are left as they are."""
    a_rows, K, E, N, R = _need_grouped(a, sa, w, sw, offsets, in_rows)
    dev = a.device
    if out_rows is not None:
        _need(out_rows, torch.int32, (R,), "out_rows", dev)
    if out is None:
        out = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, (out.shape[0], N), "out", dev)
    if R == 0:
        return out
    ws = _stream_workspace(moe_grouped_fp8_workspace(R, K, N, E), dev, workspace)
    _check(lib.fme_moe_grouped_gemm_fp8(a.data_ptr(), sa.data_ptr(), a_rows, w.data_ptr(), sw.data_ptr(),
                                        offsets.data_ptr(), _addr(in_rows), _addr(out_rows), R, K, N, E,
                                        out.data_ptr(), out.shape[0], ws.buf.data_ptr(), ws.nbytes,
                                        _launch_stream(dev)))
    return out


def moe_prompt_workspaces(T, H, I, E, top_k, device):
    """The workspaces of moe_prompt_fp8 (routing, gate/up and down product) for up to T tokens."""
    R = T * top_k
    return (Workspace(moe_route_workspace(T, E, top_k), device),
            Workspace(moe_grouped_fp8_workspace(R, H, 2 * I, E), device),
            Workspace(moe_grouped_fp8_workspace(R, I, H, E), device))


def moe_prompt_fp8(xq, sx, logits, bias, w13, s13, w2, s2, top_k, limit, scale, ue8m0, shared_out=None,
                   workspaces=None):
    """The routed FP8 experts of a prompt of T tokens, combined: moe_route, moe_grouped_swiglu_fp8 on the tokens' rows,
    moe_grouped_gemm_fp8 back to route order and moe_finalize (with shared_out [T, H] BF16 added when given).

    xq [T, H] uint8 E4M3 and sx [T, H/128] float32 as add_rmsnorm_fp8 returns them; the rest as moe_routed_fp8, whose
    weights these are, and whose shapes are checked alike. Returns (y [T, H] BF16, ids, weights); no tokens give empty
    ones. Without workspaces (moe_prompt_workspaces) the binding's kept ones serve, whose device errors
    kept_workspace_error reads; a graph that is to report its errors needs workspaces of the caller's."""
    T, H = xq.shape
    E, I = logits.shape[-1], w2.shape[-1]
    for t, shape, name in ((sx, (T, H // 128), "sx"), (logits, (T, E), "logits"), (bias, (E,), "bias"),
                           (w13, (E, 2 * I, H), "w13"), (w2, (E, H, I), "w2"), (shared_out, (T, H), "shared_out")):
        if t is not None and t.shape != shape:
            raise ValueError(f"{name}: expected {shape}, got {tuple(t.shape)}")
        if t is not None and t.device != xq.device:
            raise ValueError(f"{name}: on {t.device}, the other operands on {xq.device}")
    ws = workspaces or (None, None, None)
    ids, weights, offsets, rows, tokens = moe_route(logits, bias, top_k, scale, workspace=ws[0])
    hq, sh = moe_grouped_swiglu_fp8(xq, sx, w13, s13, offsets, in_rows=tokens, limit=limit, ue8m0=ue8m0,
                                    workspace=ws[1])
    out = moe_grouped_gemm_fp8(hq, sh, w2, s2, offsets, out_rows=rows, workspace=ws[2])
    if xq.shape[0] == 0:
        return out, ids, weights
    return moe_finalize(out, weights, shared_out), ids, weights


def moe_routed_nvfp4_workspace(M, H, N, L, top_k):
    return lib.fme_moe_routed_nvfp4_workspace(M, H, N, L, top_k)


def moe_routed_nvfp4(x, topk_ids, topk_weights, w13, s13, w2, s2, e0, limit=float("inf"), y=None,
                     workspace=None):
    """NVFP4 slot MoE over local experts [e0, e0 + L) (fme_moe_routed_nvfp4).
    w13 [L, 2N, H/2] uint8 packed E2M1 (gate rows then up rows), s13 [L, 2N, H/16]
    uint8 UE4M3, w2 [L, H, N/2], s2 [L, H, N/16]. Returns y [M, H] bf16."""
    M, H = x.shape
    L, n2, _ = w13.shape
    N = n2 // 2
    top_k = topk_ids.shape[1]
    dev = x.device
    _need(x, torch.bfloat16, (M, H), "x")
    _need(topk_ids, torch.int32, (M, top_k), "topk_ids")
    _need(topk_weights, torch.float32, (M, top_k), "topk_weights")
    _need(w13, torch.uint8, (L, 2 * N, H // 2), "w13")
    _need(s13, torch.uint8, (L, 2 * N, H // 16), "s13")
    _need(w2, torch.uint8, (L, H, N // 2), "w2")
    _need(s2, torch.uint8, (L, H, N // 16), "s2")
    if y is None:
        y = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    need = moe_routed_nvfp4_workspace(M, H, N, L, top_k)
    ws = _workspace(need, dev, workspace)
    _check(lib.fme_moe_routed_nvfp4(_ptr(x), _ptr(topk_ids), _ptr(topk_weights), _ptr(w13), _ptr(s13), _ptr(w2),
                                    _ptr(s2), M, H, N, L, int(e0), top_k, float(limit), _ptr(y), ws.ptr(),
                                    ws.nbytes, _stream(dev)))
    return y


def moe_layer_nvfp4(x, logits, bias, w13, s13, w2, s2, e0, top_k, scale=1.0, limit=float("inf"), y=None,
                    workspace=None):
    """NVFP4 slot MoE with the routing fused in (fme_moe_layer_nvfp4): logits [M, E]
    FP32 or BF16 and bias [E] FP32 pick top_k of E experts per token; the slots of the
    local experts [e0, e0 + L) run as in moe_routed_nvfp4. Returns (y, ids, weights)."""
    M, H = x.shape
    E = logits.shape[1]
    L, n2, _ = w13.shape
    N = n2 // 2
    dev = x.device
    _need(x, torch.bfloat16, (M, H), "x")
    if logits.dtype == torch.float32:
        dt = FME_F32
    elif logits.dtype == torch.bfloat16:
        dt = FME_BF16
    else:
        raise ValueError("logits must be float32 or bfloat16")
    _need(logits, logits.dtype, (M, E), "logits")
    _need(bias, torch.float32, (E,), "bias")
    _need(w13, torch.uint8, (L, 2 * N, H // 2), "w13")
    _need(s13, torch.uint8, (L, 2 * N, H // 16), "s13")
    _need(w2, torch.uint8, (L, H, N // 2), "w2")
    _need(s2, torch.uint8, (L, H, N // 16), "s2")
    if y is None:
        y = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    ids = torch.empty(M, top_k, dtype=torch.int32, device=dev)
    weights = torch.empty(M, top_k, dtype=torch.float32, device=dev)
    need = moe_routed_nvfp4_workspace(M, H, N, L, top_k)
    ws = _workspace(need, dev, workspace)
    _check(lib.fme_moe_layer_nvfp4(_ptr(x), _ptr(logits), dt, _ptr(bias), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2),
                                   M, H, N, L, E, int(e0), int(top_k), float(scale), float(limit), _ptr(y),
                                   _ptr(ids), _ptr(weights), ws.ptr(), ws.nbytes, _stream(dev)))
    return y, ids, weights


def sm_count():
    return lib.fme_sm_count()
