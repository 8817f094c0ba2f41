"""Thin Python binding of libhla2 (the C ABI in include/hla2.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, checks type/shape/contiguity, and passes raw device pointers,
sizes and the current CUDA stream to the C entry point of the same name.  All
computation happens in the library's CUDA kernels.  If ``libhla2.so`` is
missing or cannot be loaded, every call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhla2.so")

HLA2_OK = 0
HLA2_ERR_INVALID = -1
HLA2_ERR_UNSUPPORTED = -2
HLA2_ERR_WORKSPACE = -3
HLA2_ERR_LAUNCH = -4
HLA2_ERR_DEVICE = -5
HLA2_DTYPE_F32 = 0
HLA2_DTYPE_BF16 = 1

_lock = threading.Lock()
_lib: ctypes.CDLL | None = None


class HLA2Error(RuntimeError):
    def __init__(self, code: int, where: str, detail: str):
        super().__init__(f"{where} failed with status {code}: {detail}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libhla2.so (built in-tree by ``higher_order_linear_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libhla2.so not built ({LIB_PATH}); run higher_order_linear_gb300.build.build()")
            L = ctypes.CDLL(LIB_PATH)
            vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            L.hla2_forward_workspace.argtypes = [i, i, i, i, i, i]
            L.hla2_forward_workspace.restype = sz
            L.hla2_forward_plan.argtypes = [i, i, i, i, ctypes.POINTER(i), ctypes.POINTER(i), ctypes.POINTER(i)]
            L.hla2_forward_plan.restype = i
            L.hla2_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp, vp]
            L.hla2_forward.restype = i
            L.hla2_step.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, vp]
            L.hla2_step.restype = i
            L.hla2_chunk_summaries.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
            L.hla2_chunk_summaries.restype = i
            L.hla2_scan.argtypes = [vp, vp, i, i, i, i, i, vp]
            L.hla2_scan.restype = i
            L.hla2_last_error_detail.argtypes = [ctypes.c_char_p, sz]
            L.hla2_last_error_detail.restype = i
            L.hla2_device_status.argtypes = [vp]
            L.hla2_device_status.restype = i
            L.hla2_selftest_wait_runout.argtypes = [vp, i, vp]
            L.hla2_selftest_wait_runout.restype = i
            L.hla2_profile_enable.argtypes = [i]
            L.hla2_profile_enable.restype = i
            L.hla2_profile_read.argtypes = [ctypes.POINTER(ctypes.c_float), i, ctypes.POINTER(i),
                                            ctypes.POINTER(ctypes.c_longlong)]
            L.hla2_profile_read.restype = i
            L.hla2_forward_path.argtypes = [i, i, i, i, i]
            L.hla2_forward_path.restype = i
            L.hla2_chunk_summaries_path.argtypes = [i, i, i, i]
            L.hla2_chunk_summaries_path.restype = i
            L.hla2_forward_noalloc.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
            L.hla2_forward_noalloc.restype = i
            L.hla2_forward_host_workspace.argtypes = [i, i, i, i, i, i, i]
            L.hla2_forward_host_workspace.restype = sz
            L.hla2_forward_host.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp, sz, vp]
            L.hla2_forward_host.restype = i
            L.hla2_step_pform.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, vp]
            L.hla2_step_pform.restype = i
            L.hla2_state_to_pform.argtypes = [vp, vp, i, i, i, vp]
            L.hla2_state_to_pform.restype = i
            L.hla2_ahla_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp, vp]
            L.hla2_ahla_forward.restype = i
            L.hla2_ahla_step.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, vp]
            L.hla2_ahla_step.restype = i
            L.hla2_ahla_forward_path.argtypes = [i, i, i, i, i]
            L.hla2_ahla_forward_path.restype = i
            L.hla2_unmasked_forward_path.argtypes = [i, i, i, i, i]
            L.hla2_unmasked_forward_path.restype = i
            L.hla2_decay_forward_path.argtypes = [i, i, i, i, i, ctypes.c_float]
            L.hla2_decay_forward_path.restype = i
            L.hla2_unmasked_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp, vp]
            L.hla2_unmasked_forward.restype = i
            L.hla2_unmasked_step.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, vp]
            L.hla2_unmasked_step.restype = i
            L.hla2_decay_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, ctypes.c_float, i, vp, sz, vp, vp]
            L.hla2_decay_forward.restype = i
            L.hla2_decay_step.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, ctypes.c_float, vp]
            L.hla2_decay_step.restype = i
            ll, f, pll, pi = ctypes.c_longlong, ctypes.c_float, ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(i)
            L.hla2_gated_scan_workspace.argtypes = [i, i, i, i]
            L.hla2_gated_scan_workspace.restype = sz
            L.hla2_gated_scan_carry_len.argtypes = [i, i]
            L.hla2_gated_scan_carry_len.restype = sz
            L.hla2_gated_scan.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, pll, i, i, i, i, vp, sz, vp]
            L.hla2_gated_scan.restype = i
            L.hla2_gated_scan_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, pll, i, i, i, i, vp,
                                                   sz, vp]
            L.hla2_gated_scan_backward.restype = i
            L.hla2_gated_step.argtypes = [vp, vp, vp, vp, vp, i, i, pll, i, i, i, i, vp]
            L.hla2_gated_step.restype = i
            L.hla2_linear_workspace.argtypes = [i, i, i, i, i]
            L.hla2_linear_workspace.restype = sz
            L.hla2_linear_forward.argtypes = [vp] * 8 + [i, i, i, i, i, pll, i, vp, sz, vp]
            L.hla2_linear_forward.restype = i
            L.hla2_linear_backward.argtypes = [vp] * 12 + [i, i, i, i, i, pll, i, vp, sz, vp]
            L.hla2_linear_backward.restype = i
            L.hla2_linear_step.argtypes = [vp] * 7 + [i, i, i, i, pll, i, vp]
            L.hla2_linear_step.restype = i
            L.hla2_rmsnorm.argtypes = [vp, vp, vp, vp, vp, ll, i, ll, ll, ll, ll, f, i, i, i, vp]
            L.hla2_rmsnorm.restype = i
            L.hla2_rmsnorm_q8.argtypes = [vp, vp, vp, vp, vp, vp, ll, i, ll, ll, ll, ll, f, i, i, vp]
            L.hla2_rmsnorm_q8.restype = i
            L.hla2_rmsnorm_backward_workspace.argtypes = [ll, i]
            L.hla2_rmsnorm_backward_workspace.restype = sz
            L.hla2_rmsnorm_backward.argtypes = [vp, vp, vp, vp, vp, vp, ll, i, pll, f, i, i, i, vp, sz, vp]
            L.hla2_rmsnorm_backward.restype = i
            L.hla2_groupnorm_workspace.argtypes = [ll, i, i, i, i]
            L.hla2_groupnorm_workspace.restype = sz
            L.hla2_groupnorm.argtypes = [vp] * 6 + [ll, i, i, i, pll, f, i, i, i, vp, sz, vp]
            L.hla2_groupnorm.restype = i
            L.hla2_groupnorm_backward.argtypes = [vp] * 9 + [ll, i, i, i, pll, i, i, i, vp, sz, vp]
            L.hla2_groupnorm_backward.restype = i
            L.hla2_rotary.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, pi, i, i, pll, i, vp]
            L.hla2_rotary.restype = i
            _lib = L
        return _lib


def hla2_last_error_detail() -> str:
    buf = ctypes.create_string_buffer(512)
    lib().hla2_last_error_detail(buf, 512)
    return buf.value.decode(errors="replace")


def _check(code: int, where: str) -> None:
    if code != HLA2_OK:
        raise HLA2Error(code, where, hla2_last_error_detail())


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return HLA2_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return HLA2_DTYPE_BF16
    raise ValueError(f"unsupported input dtype {t.dtype}")


def _same_device(device: torch.device, **tensors) -> None:
    """Every tensor must live on ``device`` (the first input's): the library
    launches on the current device, which the calls below make ``device``."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the inputs on {device}")


def _qkv(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor):
    """Shape, dtype and device checks shared by the forwards; returns
    (B, H, T, d, dv, dtype code).  Runs before anything touches the library."""
    if Q.dim() != 4 or K.shape != Q.shape or V.dim() != 4 or V.shape[:3] != Q.shape[:3]:
        raise ValueError("expected Q, K [B,H,T,d] and V [B,H,T,dv]")
    if not (Q.dtype == K.dtype == V.dtype):
        raise ValueError(f"Q, K, V must share a dtype (got {Q.dtype}, {K.dtype}, {V.dtype})")
    _same_device(Q.device, K=K, V=V)
    B, H, T, d = Q.shape
    return B, H, T, d, V.shape[-1], _dtype_code(Q)


def _out(O: torch.Tensor | None, shape, device: torch.device) -> torch.Tensor:
    """The caller's output tensor, checked, or a new fp32 one."""
    if O is None:
        return torch.empty(shape, device=device, dtype=torch.float32)
    if tuple(O.shape) != tuple(shape):
        raise ValueError(f"O has shape {tuple(O.shape)}, expected {tuple(shape)}")
    if O.dtype != torch.float32:
        raise ValueError(f"O must be float32, got {O.dtype}")
    if not O.is_contiguous():
        raise ValueError("O must be contiguous")
    _same_device(device, O=O)
    return O


def hla2_forward_workspace(B: int, H: int, T: int, d: int, dv: int, dtype: int) -> int:
    return int(lib().hla2_forward_workspace(B, H, T, d, dv, dtype))


def hla2_forward_plan(B: int, H: int, T: int, sm_count: int = 0):
    """The forward's segment plan: (segments per head, chunks of 128 tokens
    per segment, SM count planned for).  sm_count <= 0 plans for the current
    device, as hla2_forward does."""
    ns, ln, used = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().hla2_forward_plan(B, H, T, int(sm_count), ctypes.byref(ns), ctypes.byref(ln), ctypes.byref(used)),
           "hla2_forward_plan")
    return int(ns.value), int(ln.value), int(used.value)


def record_len(d: int, dv: int) -> int:
    return d * d + 2 * d * dv + 2 * d


def _cuda_device(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _forward(entry: str, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor | None,
             normalized: bool, workspace: torch.Tensor | None, state_out: torch.Tensor | None, stream,
             state_len: int | None, gamma: float | None = None) -> torch.Tensor:
    """Common marshalling of the four forwards (same C signature, plus gamma
    before the dtype for the decayed one).  Every check runs before the
    library is touched; the call itself runs with Q's device current, so the
    default stream and the library's per-device state are that device's."""
    B, H, T, d, dv, code = _qkv(Q, K, V)
    O = _out(O, (B, H, T, dv), Q.device)
    if state_out is not None:
        if state_len is None or state_out.numel() != B * H * state_len:
            raise ValueError(f"state_out must hold B*H = {B * H} states of {state_len} floats")
    _same_device(Q.device, workspace=workspace, state_out=state_out)
    dev = _cuda_device(Q, "Q")
    with torch.cuda.device(dev):
        need = hla2_forward_workspace(B, H, T, d, dv, code)
        if workspace is None:
            workspace = torch.empty(max(need, 16), device=dev, dtype=torch.uint8)
        sptr = _dev(state_out, "state_out", torch.float32) if state_out is not None else None
        args = [_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(O, "O", torch.float32),
                B, H, T, d, dv, int(bool(normalized))]
        if gamma is not None:
            args.append(float(gamma))
        args += [code, _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), sptr,
                 _stream(stream)]
        rc = getattr(lib(), entry)(*args)
    _check(rc, entry)
    return O


def hla2_forward(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor | None = None,
                 normalized: bool = False, workspace: torch.Tensor | None = None,
                 state_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Masked second-order HLA forward.  Q, K [B,H,T,d], V [B,H,T,dv] (fp32 or
    bf16, same dtype, same device) -> O [B,H,T,dv] fp32.  ``state_out``
    [B*H, record] fp32 receives the final decode state S|C|G|m|h if given."""
    return _forward("hla2_forward", Q, K, V, O, normalized, workspace, state_out, stream, record_len(*_dims(Q, V)))


def _dims(Q: torch.Tensor, V: torch.Tensor):
    return (Q.shape[-1] if Q.dim() else 0), (V.shape[-1] if V.dim() else 0)


def hla2_forward_noalloc(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor | None = None,
                         normalized: bool = False, stream=None) -> torch.Tensor:
    """hla2_forward for callers that cannot allocate device scratch: the
    library uses its own fixed 64 MiB device array instead of a workspace
    (larger problems raise).  Only O is allocated here, and only when the
    caller passes none.  The arguments are checked as for hla2_forward
    before anything is launched."""
    B, H, T, d, dv, code = _qkv(Q, K, V)
    O = _out(O, (B, H, T, dv), Q.device)
    dev = _cuda_device(Q, "Q")
    with torch.cuda.device(dev):
        rc = lib().hla2_forward_noalloc(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(O, "O", torch.float32),
                                        B, H, T, d, dv, int(bool(normalized)), code, _stream(stream))
    _check(rc, "hla2_forward_noalloc")
    return O


def _host(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def hla2_forward_host_workspace(B: int, H: int, T: int, d: int, dv: int, dtype: int, heads_per_group: int = 0) -> int:
    return int(lib().hla2_forward_host_workspace(B, H, T, d, dv, dtype, heads_per_group))


def hla2_forward_host(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor | None = None,
                      normalized: bool = False, heads_per_group: int = 0, dev: torch.Tensor | None = None,
                      stream=None, device=None) -> torch.Tensor:
    """Masked forward on host tensors (pinned for overlap): Q, K [B,H,T,d],
    V [B,H,T,dv] on the CPU -> O [B,H,T,dv] fp32 on the CPU.  The library
    copies groups of heads in, runs the forward and copies O out as a
    pipeline on the GPU that holds ``dev`` (else ``device``, else the current
    one), which is made current for the call; O is complete once ``stream``
    (that device's current stream by default) has been synchronised.  ``dev``
    is the device buffer of hla2_forward_host_workspace(...) bytes (allocated
    here when None)."""
    if Q.dim() != 4 or K.shape != Q.shape or V.dim() != 4 or V.shape[:3] != Q.shape[:3]:
        raise ValueError("expected Q, K [B,H,T,d] and V [B,H,T,dv]")
    if not (Q.dtype == K.dtype == V.dtype):
        raise ValueError("Q, K, V must share a dtype")
    B, H, T, d = Q.shape
    dv = V.shape[-1]
    code = _dtype_code(Q)
    if O is None:
        O = torch.empty((B, H, T, dv), dtype=torch.float32, pin_memory=Q.is_pinned())
    elif O.shape != (B, H, T, dv):
        raise ValueError("O has the wrong shape")
    if dev is not None:
        gpu = _cuda_device(dev, "dev")
        if device is not None and torch.device(device) != gpu:
            raise ValueError(f"dev is on {gpu}, device is {device}")
    else:
        gpu = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(gpu):
        need = hla2_forward_host_workspace(B, H, T, d, dv, code, heads_per_group)
        if dev is None:
            dev = torch.empty(max(need, 256), dtype=torch.uint8, device=gpu)
        rc = lib().hla2_forward_host(_host(Q, "Q"), _host(K, "K"), _host(V, "V"), _host(O, "O", torch.float32),
                                     B, H, T, d, dv, int(bool(normalized)), code, int(heads_per_group),
                                     _dev(dev, "dev"), dev.numel() * dev.element_size(), _stream(stream))
    _check(rc, "hla2_forward_host")
    return O


def _step(entry: str, state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
          o: torch.Tensor | None, normalized: bool, stream, state_len_fn, gamma: float | None = None) -> torch.Tensor:
    """Common marshalling of the decode steps: state [n, state_len] fp32
    (updated in place), q, k [n, d], v [n, dv] fp32 -> o [n, dv] fp32."""
    if q.dim() != 2 or k.shape != q.shape or v.dim() != 2 or v.shape[0] != q.shape[0]:
        raise ValueError(f"{entry}: expected q, k [n,d] and v [n,dv]")
    n, d = q.shape
    dv = v.shape[-1]
    if state.numel() != n * state_len_fn(d, dv):
        raise ValueError(f"{entry}: state must hold n = {n} states of {state_len_fn(d, dv)} floats")
    if o is not None and tuple(o.shape) != (n, dv):
        raise ValueError(f"{entry}: o has shape {tuple(o.shape)}, expected {(n, dv)}")
    _same_device(q.device, k=k, v=v, state=state, o=o)
    dev = _cuda_device(q, "q")
    with torch.cuda.device(dev):
        if o is None:
            o = torch.empty((n, dv), device=dev, dtype=torch.float32)
        args = [_dev(state, "state", torch.float32), _dev(q, "q", torch.float32), _dev(k, "k", torch.float32),
                _dev(v, "v", torch.float32), _dev(o, "o", torch.float32), n, d, dv, int(bool(normalized))]
        if gamma is not None:
            args.append(float(gamma))
        args.append(_stream(stream))
        rc = getattr(lib(), entry)(*args)
    _check(rc, entry)
    return o


def hla2_step(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
              o: torch.Tensor | None = None, normalized: bool = False, stream=None) -> torch.Tensor:
    """One decode step for n heads.  state [n, record] fp32 (S|C|G|m|h,
    updated in place), q, k [n, d], v [n, dv] fp32 -> o [n, dv] fp32."""
    return _step("hla2_step", state, q, k, v, o, normalized, stream, record_len)


def pform_record_len(d: int, dv: int) -> int:
    return d * d + d * dv + d


def hla2_step_pform(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    o: torch.Tensor | None = None, normalized: bool = False, stream=None) -> torch.Tensor:
    """Decode step on the compact P-form state [n, d*d + d*dv + d] (S | P | p)."""
    return _step("hla2_step_pform", state, q, k, v, o, normalized, stream, pform_record_len)


def hla2_state_to_pform(gstate: torch.Tensor, d: int, dv: int, pstate: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """S|C|G|m|h decode states -> S|P|p (P = S C - G, p = S m - h)."""
    n = gstate.numel() // record_len(d, dv)
    if gstate.numel() != n * record_len(d, dv):
        raise ValueError("gstate size is not a whole number of records")
    if pstate is not None and pstate.numel() != n * pform_record_len(d, dv):
        raise ValueError(f"pstate must hold n = {n} states of {pform_record_len(d, dv)} floats")
    _same_device(gstate.device, pstate=pstate)
    dev = _cuda_device(gstate, "gstate")
    with torch.cuda.device(dev):
        if pstate is None:
            pstate = torch.empty((n, pform_record_len(d, dv)), device=dev, dtype=torch.float32)
        rc = lib().hla2_state_to_pform(_dev(gstate, "gstate", torch.float32), _dev(pstate, "pstate", torch.float32),
                                       n, d, dv, _stream(stream))
    _check(rc, "hla2_state_to_pform")
    return pstate


def hla2_chunk_summaries(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, L: int,
                         summ: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[B,H,N,record] fp32 chunk summaries S|C|m|G|h, N = ceil(T/L)."""
    B, H, T, d, dv, code = _qkv(Q, K, V)
    if L <= 0:
        raise ValueError("chunk length L must be positive")
    N = (T + L - 1) // L
    if summ is not None and summ.numel() != B * H * N * record_len(d, dv):
        raise ValueError(f"summ must hold B*H*N = {B * H * N} records of {record_len(d, dv)} floats")
    _same_device(Q.device, summ=summ)
    dev = _cuda_device(Q, "Q")
    with torch.cuda.device(dev):
        if summ is None:
            summ = torch.empty((B, H, N, record_len(d, dv)), device=dev, dtype=torch.float32)
        rc = lib().hla2_chunk_summaries(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(summ, "summ", torch.float32),
                                        B, H, T, d, dv, int(L), code, _stream(stream))
    _check(rc, "hla2_chunk_summaries")
    return summ


def hla2_scan(summ: torch.Tensor, d: int, dv: int, prefix: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Exclusive scan of [B,H,N,record] summaries with the semidirect combine."""
    if summ.dim() != 4:
        raise ValueError("summ must be [B,H,N,record]")
    B, H, N, R = summ.shape
    if R != record_len(d, dv):
        raise ValueError("record length does not match d, dv")
    if prefix is not None and tuple(prefix.shape) != tuple(summ.shape):
        raise ValueError("prefix must have the shape of summ")
    _same_device(summ.device, prefix=prefix)
    dev = _cuda_device(summ, "summ")
    with torch.cuda.device(dev):
        if prefix is None:
            prefix = torch.empty_like(summ)
        rc = lib().hla2_scan(_dev(summ, "summ", torch.float32), _dev(prefix, "prefix", torch.float32),
                             B, H, N, d, dv, _stream(stream))
    _check(rc, "hla2_scan")
    return prefix


def hla2_device_status(stream=None) -> int:
    return int(lib().hla2_device_status(_stream(stream)))


def hla2_selftest_wait_runout(flag: torch.Tensor, wait_us: int, stream=None) -> None:
    """Runs the library's wait run-out on purpose (see include/hla2.h); flag
    is a CUDA int32 tensor of one element that receives 0 when the wait gave
    up.  Read the status afterwards with hla2_device_status."""
    if not (isinstance(flag, torch.Tensor) and flag.is_cuda and flag.dtype == torch.int32 and flag.numel() >= 1):
        raise ValueError("flag must be a CUDA int32 tensor with at least one element")
    with torch.cuda.device(flag.device):
        _check(lib().hla2_selftest_wait_runout(ctypes.c_void_p(flag.data_ptr()), int(wait_us), _stream(stream)),
               "hla2_selftest_wait_runout")


def hla2_profile_enable(on: bool = True) -> None:
    _check(lib().hla2_profile_enable(int(bool(on))), "hla2_profile_enable")


def hla2_profile_read():
    """(phase_ms[3], profiled forwards, kernels launched) since the last read;
    phases are segment summaries, scan, segment outputs."""
    ms = (ctypes.c_float * 3)()
    nf = ctypes.c_int(0)
    nl = ctypes.c_longlong(0)
    _check(lib().hla2_profile_read(ms, 3, ctypes.byref(nf), ctypes.byref(nl)), "hla2_profile_read")
    return [float(x) for x in ms], int(nf.value), int(nl.value)


# ------------------------------------------------------------------ AHLA ----
def ahla_state_len(d: int, dv: int) -> int:
    """AHLA decode state per head: P (d x dv) | E (d x dv) | m (d) | n (d)."""
    return 2 * d * dv + 2 * d


def hla2_ahla_forward(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor | None = None,
                      normalized: bool = False, workspace: torch.Tensor | None = None,
                      state_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Masked AHLA forward (o_t = sum_{j<=i<=t} (q_t.k_i)(q_i.k_j) v_j).
    Shapes and dtypes as for hla2_forward; ``state_out`` [B*H, 2*d*dv + 2*d]
    fp32 receives the final P|E|m|n state if given."""
    return _forward("hla2_ahla_forward", Q, K, V, O, normalized, workspace, state_out, stream,
                    ahla_state_len(*_dims(Q, V)))


def hla2_ahla_step(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   o: torch.Tensor | None = None, normalized: bool = False, stream=None) -> torch.Tensor:
    """One AHLA decode step for n heads: state [n, 2*d*dv + 2*d] fp32 (P|E|m|n,
    updated in place), q, k [n, d], v [n, dv] fp32 -> o [n, dv] fp32."""
    return _step("hla2_ahla_step", state, q, k, v, o, normalized, stream, ahla_state_len)


# -------------------------------------------------------------- unmasked ----
def unmasked_state_len(d: int, dv: int) -> int:
    """Unmasked decode state per head: S (d x d) | C (d x dv) | m (d)."""
    return d * d + d * dv + d


def hla2_unmasked_forward(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor | None = None,
                          normalized: bool = False, workspace: torch.Tensor | None = None,
                          state_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Unmasked second-order forward o_t = q_t^T S_t C_t.  Shapes and dtypes
    as for hla2_forward; ``state_out`` [B*H, d*d + d*dv + d] fp32 receives the
    final S|C|m if given."""
    return _forward("hla2_unmasked_forward", Q, K, V, O, normalized, workspace, state_out, stream,
                    unmasked_state_len(*_dims(Q, V)))


def hla2_unmasked_step(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       o: torch.Tensor | None = None, normalized: bool = False, stream=None) -> torch.Tensor:
    """One unmasked decode step: state [n, d*d + d*dv + d] fp32 (S|C|m, in place)."""
    return _step("hla2_unmasked_step", state, q, k, v, o, normalized, stream, unmasked_state_len)


# ----------------------------------------------------------------- decay ----
def hla2_decay_forward(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, gamma: float,
                       O: torch.Tensor | None = None, normalized: bool = False,
                       workspace: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """Decayed masked forward, o_t = sum_{i<=j<=t} gamma^{2t-i-j} (q_t.k_i)(k_i.q_j) v_j.
    Shapes and dtypes as for hla2_forward; ``state_out`` [B*H, d*d + d*dv + d]
    fp32 receives the final compact state S|P|p if given."""
    return _forward("hla2_decay_forward", Q, K, V, O, normalized, workspace, state_out, stream,
                    pform_record_len(*_dims(Q, V)), gamma=gamma)


def hla2_decay_step(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gamma: float,
                    o: torch.Tensor | None = None, normalized: bool = False, stream=None) -> torch.Tensor:
    """One decayed decode step on the compact state [n, d*d + d*dv + d] (S|P|p, in place)."""
    return _step("hla2_decay_step", state, q, k, v, o, normalized, stream, pform_record_len, gamma=gamma)


# ------------------------------------------------ around the attention layer ----
# The gated linear recurrence, the root-mean-square norm and the rotary
# positions.  Their tensors may be strided (the last dimension contiguous).
# A decoding step makes these calls on a few kilobytes, where the call itself is
# the cost: the step, the norms and the rotary call first ask in one expression
# whether the arguments are the ordinary ones (dense, outputs not given, a gate for
# each channel), and only otherwise go through the checks one by one.
_GATE_FORMS = {"sigmoid": 0, "decay": 1}
_CODES = {torch.float32: HLA2_DTYPE_F32, torch.bfloat16: HLA2_DTYPE_BF16}
_F32 = torch.float32


@functools.lru_cache(maxsize=256)
def _longs(*values):
    """Strides as the C entries take them (read only: the same values share one array)."""
    return (ctypes.c_longlong * len(values))(*values)


@functools.lru_cache(maxsize=64)
def _ints(*values):
    return (ctypes.c_int * len(values))(*values)


class _NoGuard:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NO_GUARD = _NoGuard()


def _guard(dev: torch.device, stream):
    """Makes ``dev`` current, and ``stream`` (when given) too, so that what the
    call allocates belongs to the stream it is used on."""
    if stream is None:
        return _NO_GUARD if torch._C._cuda_getDevice() == dev.index else torch.cuda.device(dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return torch.cuda.stream(stream)


def _raw(dev: torch.device, stream) -> int:
    """The stream's handle; the current stream of ``dev`` by default."""
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else _stream(stream)


def _operand(t, name: str, device=None, dtype=None, shape=None, dense=False) -> None:
    """Checks of one operand, before anything is allocated or launched."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the inputs on {device}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _last_dense(t: torch.Tensor, name: str) -> None:
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _no_overlap(t: torch.Tensor, name: str) -> None:
    """An output must not hold one element in two places."""
    if any(st == 0 and n > 1 for st, n in zip(t.stride(), t.shape)):
        raise ValueError(f"{name} must not be an expanded tensor")


def _output(t, name: str, dev, dtype, shape) -> None:
    _operand(t, name, dev, dtype, shape)
    if t.dim():
        _last_dense(t, name)
    _no_overlap(t, name)


def _out_code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported output dtype {dtype}")
    return code


def _like(t: torch.Tensor, dtype=None) -> torch.Tensor:
    """An output in t's memory order, its last dimension contiguous (t's elements may overlap, as in
    sliding windows: then the order is not always t's)."""
    o = torch.empty_like(t, dtype=dtype)
    return o if o.stride(-1) == 1 or t.shape[-1] == 1 else torch.empty(t.shape, device=t.device, dtype=o.dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def hla2_gated_scan_workspace(B: int, H: int, T: int, d: int) -> int:
    return int(lib().hla2_gated_scan_workspace(B, H, T, d))


def hla2_gated_scan_carry_len(T: int, d: int) -> int:
    """Floats per head of the ``carry`` that a forward keeps for its backward."""
    return int(lib().hla2_gated_scan_carry_len(T, d))


def _gated_inputs(X, G, form, reset):
    """Checks shared by the scan and its backward; returns (B, H, T, d, dtype code, form code, shared)."""
    _operand(X, "X")
    _operand(G, "G")
    if X.dim() != 4 or (G.shape != X.shape and G.shape != X.shape[:3]):
        raise ValueError("expected X [B,H,T,d] and G [B,H,T,d] or [B,H,T]")
    if X.dtype != G.dtype:
        raise ValueError(f"X and G must share a dtype (got {X.dtype}, {G.dtype})")
    code = _dtype_code(X)
    if form not in _GATE_FORMS:
        raise ValueError(f"unknown gate form {form!r}: one of {sorted(_GATE_FORMS)}")
    _operand(G, "G", X.device)
    B, H, T, d = X.shape
    shared = G.dim() == 3
    _last_dense(X, "X")
    if not shared:
        _last_dense(G, "G")
    if reset is not None:
        if not isinstance(reset, torch.Tensor) or reset.dtype not in (torch.bool, torch.uint8):
            raise ValueError("reset must be a bool or uint8 tensor")
        _operand(reset, "reset", X.device, shape=(B, T), dense=True)
    return B, H, T, d, code, _GATE_FORMS[form], shared


def _gated_optional(dev, B, H, T, d, carry, workspace, **states):
    for name, t in states.items():
        if t is not None:
            _operand(t, name, dev, _F32, (B, H, d), dense=True)
    if carry is not None:
        _operand(carry, "carry", dev, _F32, (B, H, hla2_gated_scan_carry_len(T, d)), dense=True)
    if workspace is not None:
        _operand(workspace, "workspace", dev, dense=True)


def _gated_work(L, workspace, B, H, T, d, dev):
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    need = L.hla2_gated_scan_workspace(B, H, T, d)
    return (torch.empty(need, device=dev, dtype=torch.uint8) if need else None), need


def hla2_gated_scan(X: torch.Tensor, G: torch.Tensor, O: torch.Tensor | None = None, form: str = "sigmoid",
                    reset: torch.Tensor | None = None, state_in: torch.Tensor | None = None,
                    state_out: torch.Tensor | None = None, carry: torch.Tensor | None = None,
                    out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t along the tokens of each
    head: X [B,H,T,d], G [B,H,T,d] or [B,H,T] (one gate for a head's channels),
    fp32 or bf16 -> O [B,H,T,d] of ``out_dtype`` (or O's own dtype), in X's
    memory order when it is not given.

    ``form`` "sigmoid": a = sigmoid(G), u = (1 - a) X;  "decay": a = G, u = X.
    ``reset`` [B,T] bool: a document begins there (h_{t-1} counts as zero).
    ``state_in`` / ``state_out`` [B,H,d] fp32: h before and after (one tensor may be both).
    ``carry`` [B,H,hla2_gated_scan_carry_len(T, d)] fp32 keeps what
    hla2_gated_scan_backward needs."""
    B, H, T, d, code, fcode, shared = _gated_inputs(X, G, form, reset)
    dev = X.device
    if O is not None:
        _output(O, "O", dev, None, X.shape)
        out_dtype = O.dtype
    ocode = _out_code(out_dtype)
    if not (state_in is state_out is carry is workspace is None):
        _gated_optional(dev, B, H, T, d, carry, workspace, state_in=state_in, state_out=state_out)
    _cuda_device(X, "X")
    L = _lib or lib()
    with _guard(dev, stream):
        if O is None:
            O = _like(X, out_dtype)
        workspace, nws = _gated_work(L, workspace, B, H, T, d, dev)
        rc = L.hla2_gated_scan(X.data_ptr(), G.data_ptr(), _ptr(reset), _ptr(state_in), O.data_ptr(),
                               _ptr(state_out), _ptr(carry), B, H, T, d,
                               _longs(*X.stride()[:3], *G.stride()[:3], *O.stride()[:3]), fcode, shared, code, ocode,
                               _ptr(workspace), nws, _raw(dev, stream))
    if rc:
        _check(rc, "hla2_gated_scan")
    return O


def hla2_gated_scan_backward(X: torch.Tensor, G: torch.Tensor, dO: torch.Tensor, carry: torch.Tensor,
                             form: str = "sigmoid", reset: torch.Tensor | None = None,
                             dstate_out: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                             dG: torch.Tensor | None = None, dstate_in: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None):
    """Gradients (dX, dG) of hla2_gated_scan over the same X, G, ``form`` and
    ``reset``; ``carry`` is what that call kept.  dO [B,H,T,d] is the gradient
    of O, ``dstate_out`` that of state_out; ``dstate_in`` [B,H,d] fp32 receives
    that of state_in (one tensor may be both).  A shared gate's dG [B,H,T] is summed over the channels."""
    B, H, T, d, code, fcode, shared = _gated_inputs(X, G, form, reset)
    dev = X.device
    _operand(dO, "dO", dev, shape=X.shape)
    ocode = _dtype_code(dO)
    _last_dense(dO, "dO")
    _operand(carry, "carry", dev, _F32)
    if dX is not None:
        _output(dX, "dX", dev, X.dtype, X.shape)
    if dG is not None:
        _operand(dG, "dG", dev, G.dtype, G.shape)
        if not shared:
            _last_dense(dG, "dG")
        _no_overlap(dG, "dG")
    _gated_optional(dev, B, H, T, d, carry, workspace, dstate_out=dstate_out, dstate_in=dstate_in)
    _cuda_device(X, "X")
    L = _lib or lib()
    with _guard(dev, stream):
        if dX is None:
            dX = _like(X)
        if dG is None:
            dG = torch.empty_like(G) if shared else _like(G)
        workspace, nws = _gated_work(L, workspace, B, H, T, d, dev)
        rc = L.hla2_gated_scan_backward(X.data_ptr(), G.data_ptr(), _ptr(reset), carry.data_ptr(), dO.data_ptr(),
                                        _ptr(dstate_out), dX.data_ptr(), dG.data_ptr(), _ptr(dstate_in), B, H, T, d,
                                        _longs(*X.stride()[:3], *G.stride()[:3], *dO.stride()[:3], *dX.stride()[:3],
                                              *dG.stride()[:3]), fcode, shared, code, ocode, _ptr(workspace), nws,
                                        _raw(dev, stream))
    if rc:
        _check(rc, "hla2_gated_scan_backward")
    return dX, dG


def _gated_step_checks(state, x, g, o, state_out):
    _operand(x, "x")
    if x.dim() != 2:
        raise ValueError("hla2_gated_step: expected x [n,d]")
    dev = x.device
    _operand(g, "g", dev)
    if g.shape != x.shape and g.shape != x.shape[:1]:
        raise ValueError("hla2_gated_step: expected g [n,d] or [n]")
    if g.dtype != x.dtype:
        raise ValueError(f"x and g must share a dtype (got {x.dtype}, {g.dtype})")
    _dtype_code(x)
    _last_dense(x, "x")
    if g.dim() == 2:
        _last_dense(g, "g")
    _operand(state, "state", dev, _F32, x.shape, dense=True)
    if state_out is not None:
        _operand(state_out, "state_out", dev, _F32, x.shape, dense=True)
    if o is not None:
        _output(o, "o", dev, None, x.shape)
    _cuda_device(x, "x")


def hla2_gated_step(state: torch.Tensor, x: torch.Tensor, g: torch.Tensor, o: torch.Tensor | None = None,
                    form: str = "sigmoid", out_dtype: torch.dtype = torch.float32,
                    state_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One token of the recurrence for n heads: state [n,d] fp32, x [n,d] and
    g [n,d] or [n] (fp32 or bf16) -> o [n,d].  The state is updated in place,
    or left and the new one written to ``state_out``."""
    shape, dt, dev = x.shape, x.dtype, x.device
    if not (x.is_cuda and x.is_contiguous() and len(shape) == 2 and dt in _CODES and o is None and
            g.shape == shape and g.dtype is dt and g.device == dev and g.is_contiguous() and
            state.shape == shape and state.dtype is _F32 and state.device == dev and state.is_contiguous() and
            (state_out is None or (state_out.shape == shape and state_out.dtype is _F32 and
                                   state_out.device == dev and state_out.is_contiguous()))):
        _gated_step_checks(state, x, g, o, state_out)
    fcode = _GATE_FORMS.get(form)
    if fcode is None:
        raise ValueError(f"unknown gate form {form!r}: one of {sorted(_GATE_FORMS)}")
    ocode = _out_code(out_dtype if o is None else o.dtype)
    n, d = shape
    L = _lib or lib()
    with _guard(dev, stream):
        if o is None:
            o = torch.empty(shape, device=dev, dtype=out_dtype)
        rc = L.hla2_gated_step(state.data_ptr(), x.data_ptr(), g.data_ptr(), o.data_ptr(),
                               None if state_out is None else state_out.data_ptr(), n, d,
                               _longs(x.stride(0), g.stride(0), o.stride(0)), fcode, g.dim() == 1, _CODES[dt], ocode,
                               _raw(dev, stream))
    if rc:
        _check(rc, "hla2_gated_step")
    return o


def hla2_linear_workspace(B: int, H: int, T: int, d: int, dv: int) -> int:
    return int(lib().hla2_linear_workspace(B, H, T, d, dv))


def _linear_checks(Q, K, V, gamma):
    """The checks of the linear attention's inputs, one by one."""
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        _operand(t, name, None if t is Q else Q.device)
        if t.dim() != 4:
            raise ValueError("expected Q, K [B,H,T,d] and V [B,H,T,dv]")
        _last_dense(t, name)
    if K.shape != Q.shape or V.shape[:3] != Q.shape[:3]:
        raise ValueError("expected Q, K [B,H,T,d] and V [B,H,T,dv]")
    if not (Q.dtype == K.dtype == V.dtype):
        raise ValueError(f"Q, K, V must share a dtype (got {Q.dtype}, {K.dtype}, {V.dtype})")
    _dtype_code(Q)
    _operand(gamma, "gamma", Q.device, _F32, Q.shape[1:2], dense=True)


def _linear_inputs(Q, K, V, gamma, lengths, workspace, **states):
    """Checks shared by the linear attention's forward and backward; returns (B, H, T, d, dv, dtype code)."""
    shape, vshape, dt, dev = Q.shape, V.shape, Q.dtype, Q.device
    if not (Q.is_cuda and len(shape) == len(vshape) == 4 and K.shape == shape and vshape[:3] == shape[:3] and
            dt in _CODES and K.dtype is dt and V.dtype is dt and K.device == dev and V.device == dev and
            Q.stride(3) == K.stride(3) == V.stride(3) == 1 and gamma.dtype is _F32 and gamma.shape == shape[1:2] and
            gamma.device == dev and gamma.is_contiguous()):
        _linear_checks(Q, K, V, gamma)
    B, H, T, d = shape
    dv = vshape[3]
    if lengths is not None:
        _operand(lengths, "lengths", dev, torch.int32, (B,), dense=True)
    for name, t in states.items():
        if t is not None:
            _operand(t, name, dev, _F32, (B, H, d, dv), dense=True)
    if workspace is not None:
        _operand(workspace, "workspace", dev, dense=True)
    return B, H, T, d, dv, _CODES[dt]


@functools.lru_cache(maxsize=256)
def _linear_need(device, B, H, T, d, dv):
    """The workspace's bytes, asked once for each size on a device (its SM count is part of the answer)."""
    return lib().hla2_linear_workspace(B, H, T, d, dv)


def _linear_work(workspace, B, H, T, d, dv, dev):
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    need = _linear_need(dev.index, B, H, T, d, dv)
    return (torch.empty(need, device=dev, dtype=torch.uint8) if need else None), need


def hla2_linear_forward(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, gamma: torch.Tensor,
                        O: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                        state_in: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """First-order linear attention with a decay for each head,
    S_t = gamma_h S_{t-1} + k_t v_t^T, o_t = S_t^T q_t: Q, K [B,H,T,d], V
    [B,H,T,dv] fp32 or bf16 (the last dimension contiguous), gamma [H] fp32 in
    [0, 1] -> O [B,H,T,dv] of the inputs' dtype, in V's memory order when it is
    not given.

    ``lengths`` [B] int32: the tokens of each sequence; what stands behind them is
    not used and O is left as it was there (zeros when it is not given).
    ``state_in`` / ``state_out`` [B,H,d,dv] fp32: S before and after (one tensor may be both);
    decoding goes on with hla2_linear_step."""
    B, H, T, d, dv, code = _linear_inputs(Q, K, V, gamma, lengths, workspace, state_in=state_in, state_out=state_out)
    dev = _cuda_device(Q, "Q")
    if O is not None:
        _output(O, "O", dev, Q.dtype, V.shape)
    L = _lib or lib()
    with _guard(dev, stream):
        if O is None:
            O = _like(V) if lengths is None else _like(V).zero_()
        workspace, nws = _linear_work(workspace, B, H, T, d, dv, dev)
        rc = L.hla2_linear_forward(Q.data_ptr(), K.data_ptr(), V.data_ptr(), gamma.data_ptr(), _ptr(lengths),
                                   _ptr(state_in), O.data_ptr(), _ptr(state_out), B, H, T, d, dv,
                                   _longs(*Q.stride()[:3], *K.stride()[:3], *V.stride()[:3], *O.stride()[:3]), code,
                                   _ptr(workspace), nws, _raw(dev, stream))
    if rc:
        _check(rc, "hla2_linear_forward")
    return O


def hla2_linear_backward(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, gamma: torch.Tensor, dO: torch.Tensor,
                         dQ: torch.Tensor | None = None, dK: torch.Tensor | None = None,
                         dV: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                         state_in: torch.Tensor | None = None, dstate_out: torch.Tensor | None = None,
                         dstate_in: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients (dQ, dK, dV) of hla2_linear_forward over the same Q, K, V, gamma,
    ``lengths`` and ``state_in``.  dO [B,H,T,dv] is the gradient of O,
    ``dstate_out`` that of state_out; ``dstate_in`` [B,H,d,dv] fp32 receives that of
    state_in (it may be dstate_out).  Behind a sequence's end the gradients are zero.
    gamma is not differentiated."""
    B, H, T, d, dv, code = _linear_inputs(Q, K, V, gamma, lengths, workspace, state_in=state_in,
                                          dstate_out=dstate_out, dstate_in=dstate_in)
    dev = _cuda_device(Q, "Q")
    _operand(dO, "dO", dev, Q.dtype, V.shape)
    _last_dense(dO, "dO")
    for name, t, like in (("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, V)):
        if t is not None:
            _output(t, name, dev, Q.dtype, like.shape)
    L = _lib or lib()
    with _guard(dev, stream):
        dQ = _like(Q) if dQ is None else dQ
        dK = _like(K) if dK is None else dK
        dV = _like(V) if dV is None else dV
        workspace, nws = _linear_work(workspace, B, H, T, d, dv, dev)
        rc = L.hla2_linear_backward(Q.data_ptr(), K.data_ptr(), V.data_ptr(), gamma.data_ptr(), _ptr(lengths),
                                    _ptr(state_in), dO.data_ptr(), _ptr(dstate_out), dQ.data_ptr(), dK.data_ptr(),
                                    dV.data_ptr(), _ptr(dstate_in), B, H, T, d, dv,
                                    _longs(*(st for t in (Q, K, V, dO, dQ, dK, dV) for st in t.stride()[:3])), code,
                                    _ptr(workspace), nws, _raw(dev, stream))
    if rc:
        _check(rc, "hla2_linear_backward")
    return dQ, dK, dV


def _linear_step_checks(state, q, k, v, gamma, o, state_out):
    _operand(q, "q")
    if q.dim() != 2:
        raise ValueError("hla2_linear_step: expected q, k [n,d] and v [n,dv]")
    dev = q.device
    _operand(k, "k", dev, q.dtype, q.shape)
    _operand(v, "v", dev, q.dtype)
    if v.dim() != 2 or v.shape[0] != q.shape[0]:
        raise ValueError("hla2_linear_step: expected q, k [n,d] and v [n,dv]")
    _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _last_dense(t, name)
    shape = (*q.shape, v.shape[1])
    _operand(state, "state", dev, _F32, shape, dense=True)
    if state_out is not None:
        _operand(state_out, "state_out", dev, _F32, shape, dense=True)
    _operand(gamma, "gamma", dev, _F32, dense=True)
    if gamma.dim() != 1 or not gamma.numel() or q.shape[0] % gamma.numel():
        raise ValueError("gamma must be [H] with the number of heads n a multiple of H")
    if o is not None:
        _output(o, "o", dev, q.dtype, v.shape)
    _cuda_device(q, "q")


def hla2_linear_step(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gamma: torch.Tensor,
                     o: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """One token of the linear attention for n heads: state [n,d,dv] fp32, q, k
    [n,d], v [n,dv] (fp32 or bf16), gamma [H] with n a multiple of H (head i decays
    by gamma[i % H]) -> o [n,dv] of the inputs' dtype (it may be v, but not overlap
    an input otherwise).  The state is updated in place, or left and the new one
    written to ``state_out``."""
    shape, dt, dev, ld = q.shape, q.dtype, q.device, None
    if not (q.is_cuda and q.is_contiguous() and len(shape) == 2 and dt in _CODES and o is None and
            k.shape == shape and k.dtype is dt and k.device == dev and k.is_contiguous() and
            v.dtype is dt and v.device == dev and v.is_contiguous() and len(v.shape) == 2 and
            v.shape[0] == shape[0] and state.shape == (*shape, v.shape[1]) and state.dtype is _F32 and
            state.device == dev and state.is_contiguous() and gamma.dtype is _F32 and gamma.device == dev and
            gamma.dim() == 1 and gamma.is_contiguous() and gamma.shape[0] and not shape[0] % gamma.shape[0] and
            (state_out is None or (state_out.shape == state.shape and state_out.dtype is _F32 and
                                   state_out.device == dev and state_out.is_contiguous()))):
        _linear_step_checks(state, q, k, v, gamma, o, state_out)
        ld = _longs(q.stride(0), k.stride(0), v.stride(0), v.shape[1] if o is None else o.stride(0))
    n, d = shape
    L = _lib or lib()
    with _guard(dev, stream):
        if o is None:
            o = torch.empty(v.shape, device=dev, dtype=dt)
        rc = L.hla2_linear_step(state.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), gamma.data_ptr(),
                                o.data_ptr(), None if state_out is None else state_out.data_ptr(), n, gamma.shape[0],
                                d, v.shape[1], ld, _CODES[dt],
                                _raw(dev, stream))
    if rc:
        _check(rc, "hla2_linear_step")
    return o


def _rows(t: torch.Tensor, name: str) -> int:
    """The row stride of a tensor whose leading dimensions run through its rows with one stride."""
    if t.is_contiguous():
        return t.shape[-1]
    C = t.shape[-1]
    _last_dense(t, name)
    ld, expect = None, None
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld, expect = st, st * n
        elif st == expect:
            expect = st * n
        else:
            raise ValueError(f"{name}: its rows must have one stride")
    if ld is None:
        return C
    if ld < C:
        raise ValueError(f"{name}: its rows overlap")
    return ld


def _norm_checks(X, weight, residual, eps):
    """The checks of the norms' inputs, one by one."""
    _operand(X, "X")
    if X.dim() < 1:
        raise ValueError("X must have at least one dimension")
    _dtype_code(X)
    if weight is not None:
        _operand(weight, "weight", X.device, shape=X.shape[-1:], dense=True)
        _dtype_code(weight)
    if residual is not None:
        _operand(residual, "residual", X.device, X.dtype, X.shape)
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    _rows(X, "X")
    if residual is not None:
        _rows(residual, "residual")


def _norm_inputs(X, weight, residual, eps):
    """Returns (rows, C, dtype code, weight pointer, weight dtype code, row strides of X and the residual)."""
    shape, dt, dev = X.shape, X.dtype, X.device
    if not (len(shape) and dt in _CODES and eps >= 0 and X.is_contiguous() and
            (weight is None or (weight.dtype in _CODES and weight.shape == shape[-1:] and weight.device == dev and
                                weight.is_contiguous())) and
            (residual is None or (residual.dtype is dt and residual.shape == shape and residual.device == dev and
                                  residual.is_contiguous()))):
        _norm_checks(X, weight, residual, eps)
    C = shape[-1]
    return (X.numel() // C if C else 0, C, _CODES[dt], None if weight is None else weight.data_ptr(),
            0 if weight is None else _CODES[weight.dtype], _rows(X, "X"),
            0 if residual is None else _rows(residual, "residual"))


def _norm_stream(X, residual, S):
    """The residual stream's new tensor (wanted with a residual) and its row stride."""
    if S is None:
        if residual is None:
            return None, 0
        return torch.empty(X.shape, device=X.device, dtype=X.dtype), X.shape[-1]
    return S, _rows(S, "S")


def hla2_rmsnorm(X: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                 Y: torch.Tensor | None = None, S: torch.Tensor | None = None, eps: float = 1e-6,
                 out_dtype: torch.dtype | None = None, stream=None):
    """Root-mean-square norm of the rows of t = X (+ residual):
    Y = t / sqrt(mean(t^2) + eps) * weight.  X [..., C] fp32 or bf16, weight [C].
    Returns (Y, S): Y of ``out_dtype`` (X's by default), S = t in X's dtype,
    the new residual stream (None without a residual unless S is given)."""
    rows, C, code, wptr, wcode, ldx, ldr = _norm_inputs(X, weight, residual, eps)
    dev = X.device
    if Y is not None:
        _output(Y, "Y", dev, None, X.shape)
        _rows(Y, "Y")
        out_dtype = Y.dtype
    elif out_dtype is None:
        out_dtype = X.dtype
    ocode = _out_code(out_dtype)
    if S is not None:
        _output(S, "S", dev, X.dtype, X.shape)
    _cuda_device(X, "X")
    L = _lib or lib()
    with _guard(dev, stream):
        if Y is None:
            Y = torch.empty(X.shape, device=dev, dtype=out_dtype)
        S, lds = _norm_stream(X, residual, S)
        rc = L.hla2_rmsnorm(X.data_ptr(), _ptr(residual), wptr, _ptr(S), Y.data_ptr(), rows, C, ldx, ldr, lds,
                            _rows(Y, "Y"), eps, code, wcode, ocode, _raw(dev, stream))
    if rc:
        _check(rc, "hla2_rmsnorm")
    return Y, S


def hla2_rmsnorm_q8(X: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                    Q: torch.Tensor | None = None, scale: torch.Tensor | None = None, S: torch.Tensor | None = None,
                    eps: float = 1e-6, stream=None):
    """The norm of hla2_rmsnorm with an 8-bit output: returns (Q, scale, S), Q
    [..., C] float8_e4m3fn and scale [...] fp32 with Y = Q * scale (scale =
    max|Y| / 448 of the row, 1 for a row of zeros)."""
    rows, C, code, wptr, wcode, ldx, ldr = _norm_inputs(X, weight, residual, eps)
    dev = X.device
    if Q is not None:
        _output(Q, "Q", dev, torch.float8_e4m3fn, X.shape)
        _rows(Q, "Q")
    if scale is not None:
        _operand(scale, "scale", dev, _F32, X.shape[:-1], dense=True)
    if S is not None:
        _output(S, "S", dev, X.dtype, X.shape)
    _cuda_device(X, "X")
    L = _lib or lib()
    with _guard(dev, stream):
        if Q is None:
            Q = torch.empty(X.shape, device=dev, dtype=torch.float8_e4m3fn)
        if scale is None:
            scale = torch.empty(X.shape[:-1], device=dev, dtype=_F32)
        S, lds = _norm_stream(X, residual, S)
        rc = L.hla2_rmsnorm_q8(X.data_ptr(), _ptr(residual), wptr, _ptr(S), Q.data_ptr(), scale.data_ptr(), rows, C,
                               ldx, ldr, lds, _rows(Q, "Q"), eps, code, wcode, _raw(dev, stream))
    if rc:
        _check(rc, "hla2_rmsnorm_q8")
    return Q, scale, S


def hla2_rmsnorm_backward(S: torch.Tensor, dY: torch.Tensor, weight: torch.Tensor | None = None,
                          dS: torch.Tensor | None = None, dX: torch.Tensor | None = None, eps: float = 1e-6,
                          workspace: torch.Tensor | None = None, stream=None):
    """Gradients of the norm at t = S (what the forward kept, or X without a
    residual): dX (of X and of the residual; ``dS``, the gradient that reaches
    the residual stream, is added) in S's dtype, and dW [C] fp32 (None without
    a weight)."""
    rows, C, code, wptr, wcode, lds, ldd = _norm_inputs(S, weight, dS, eps)
    dev = S.device
    _operand(dY, "dY", dev, shape=S.shape)
    ycode = _dtype_code(dY)
    ldy = _rows(dY, "dY")
    if dX is not None:
        _output(dX, "dX", dev, S.dtype, S.shape)
        _rows(dX, "dX")
    if workspace is not None:
        _operand(workspace, "workspace", dev, dense=True)
    _cuda_device(S, "S")
    L = _lib or lib()
    with _guard(dev, stream):
        if dX is None:
            dX = torch.empty(S.shape, device=dev, dtype=S.dtype)
        dW, nws = None, 0
        if weight is not None:
            dW = torch.empty((C,), device=dev, dtype=_F32)
            if workspace is None:
                workspace = torch.empty(L.hla2_rmsnorm_backward_workspace(rows, C), device=dev, dtype=torch.uint8)
            nws = workspace.numel() * workspace.element_size()
        rc = L.hla2_rmsnorm_backward(S.data_ptr(), dY.data_ptr(), wptr, _ptr(dS), dX.data_ptr(), _ptr(dW), rows, C,
                                     _longs(lds, ldy, ldd, _rows(dX, "dX")), eps, code, wcode, ycode, _ptr(workspace),
                                     nws, _raw(dev, stream))
    if rc:
        _check(rc, "hla2_rmsnorm_backward")
    return dX, dW


_ACTIVATIONS = {"none": 0, "silu": 1}


def hla2_groupnorm_workspace(N: int, L: int, C: int, groups: int, backward: bool = False) -> int:
    return int(lib().hla2_groupnorm_workspace(N, L, C, groups, int(bool(backward))))


def _group_view(t, shape):
    """Strides of samples and positions of [N, C] or [N, L, C]."""
    if t is None:
        return 0, 0
    st = t.stride()
    return (st[0], st[1]) if len(shape) == 3 else (st[0], 0)


def _group_checks(X, groups, weight, bias, gate, stats, workspace, **like):
    """The checks of the group norm's inputs, one by one."""
    _operand(X, "X")
    if X.dim() not in (2, 3):
        raise ValueError("expected X [N,C] or [N,L,C]")
    _dtype_code(X)
    dev, C = X.device, X.shape[-1]
    _last_dense(X, "X")
    if groups < 1 or C % groups:
        raise ValueError(f"groups must divide the {C} channels, got {groups}")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _operand(t, name, dev, shape=(C,), dense=True)
            _dtype_code(t)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError(f"weight and bias must share a dtype (got {weight.dtype}, {bias.dtype})")
    if gate is not None:
        _operand(gate, "gate", dev, X.dtype, X.shape)
        _last_dense(gate, "gate")
    if stats is not None:
        _operand(stats, "stats", dev, _F32, (X.shape[0], groups, 2), dense=True)
    if workspace is not None:
        _operand(workspace, "workspace", dev, dense=True)
    for name, t in like.items():
        if t is not None:
            _output(t, name, dev, X.dtype, X.shape)
    _cuda_device(X, "X")


def _group_plain(X, groups, weight, bias, gate, stats):
    """Whether all arguments are the ordinary ones: dense, weight and bias of one type."""
    shape, dt, dev = X.shape, X.dtype, X.device
    return (X.is_cuda and len(shape) in (2, 3) and dt in _CODES and X.is_contiguous() and groups >= 1 and
            not shape[-1] % groups and weight is not None and bias is not None and weight.dtype in _CODES and
            weight.dtype is bias.dtype and weight.shape == bias.shape == shape[-1:] and
            weight.device == bias.device == dev and weight.is_contiguous() and bias.is_contiguous() and
            (gate is None or (gate.dtype is dt and gate.shape == shape and gate.device == dev and
                              gate.is_contiguous())) and
            (stats is None or (stats.dtype is _F32 and stats.shape == (shape[0], groups, 2) and
                               stats.device == dev and stats.is_contiguous())))


def _activation(name) -> int:
    code = _ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r}: one of {sorted(_ACTIVATIONS)}")
    return code


@functools.lru_cache(maxsize=256)
def _group_need(device, N, P, C, groups, backward):
    """The workspace's bytes, asked once for each size on a device (its SM count is part of the answer)."""
    return lib().hla2_groupnorm_workspace(N, P, C, groups, backward)


def _group_work(workspace, N, P, C, groups, backward, dev):
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    need = _group_need(dev.index, N, P, C, groups, backward)
    return (torch.empty(need, device=dev, dtype=torch.uint8) if need else None), need


def hla2_groupnorm(X: torch.Tensor, groups: int, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                   gate: torch.Tensor | None = None, activation: str = "none", Y: torch.Tensor | None = None,
                   stats: torch.Tensor | None = None, eps: float = 1e-5, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Group norm, channels last: X [N,L,C] (statistics over a sample's L positions
    and a group's C / groups channels) or [N,C] (L = 1: the groups of each row, as
    behind an attention layer with a group for each head), fp32 or bf16 -> Y like
    X.  z = (X - mean) / sqrt(var + eps) * weight + bias;  Y = act(z), or
    z * act(gate) with a ``gate`` like X;  ``activation`` "none" or "silu".
    weight, bias [C] fp32 or bf16.  ``stats`` [N,groups,2] fp32 keeps what
    hla2_groupnorm_backward needs.  Y may be X or gate."""
    acode, strides = _activation(activation), None
    if Y is not None or workspace is not None or not _group_plain(X, groups, weight, bias, gate, stats):
        _group_checks(X, groups, weight, bias, gate, stats, workspace, Y=Y)
        strides = 0
    dev, shape = X.device, X.shape
    N, C = shape[0], shape[-1]
    P = shape[1] if len(shape) == 3 else 1
    wcode = _CODES[weight.dtype if weight is not None else bias.dtype if bias is not None else _F32]
    L = _lib or lib()
    with _guard(dev, stream):
        if Y is None:
            Y = _like(X)
        if strides is not None:
            strides = _longs(*_group_view(X, shape), *_group_view(gate, shape), *_group_view(Y, shape))
        workspace, nws = _group_work(workspace, N, P, C, groups, 0, dev)
        rc = L.hla2_groupnorm(X.data_ptr(), _ptr(weight), _ptr(bias), _ptr(gate), Y.data_ptr(), _ptr(stats), N, P, C,
                              groups, strides, eps, acode, _CODES[X.dtype], wcode, _ptr(workspace), nws, _raw(dev, stream))
    if rc:
        _check(rc, "hla2_groupnorm")
    return Y


def hla2_groupnorm_backward(X: torch.Tensor, dY: torch.Tensor, stats: torch.Tensor, weight: torch.Tensor | None = None,
                            bias: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                            activation: str = "none", dX: torch.Tensor | None = None,
                            dgate: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of hla2_groupnorm at X, with the ``stats`` [N,groups,2] that the
    forward kept and its weight, bias, gate and activation: (dX, dW, dB, dgate), dX
    and dgate in X's dtype (dgate None without a gate), dW and dB [C] fp32.  dX may
    be dY or X, dgate may be gate."""
    acode = _activation(activation)
    groups = stats.shape[1] if isinstance(stats, torch.Tensor) and stats.dim() == 3 else 0
    if not groups:
        raise ValueError("expected stats [N,groups,2]")
    strides = None
    if not (dX is dgate is workspace is None and _group_plain(X, groups, weight, bias, gate, stats) and
            dY.dtype is X.dtype and dY.shape == X.shape and dY.device == X.device and dY.is_contiguous()):
        strides = 0
        if gate is None and dgate is not None:
            raise ValueError("dgate without a gate")
        _group_checks(X, groups, weight, bias, gate, stats, workspace, dX=dX, dgate=dgate)
        _operand(dY, "dY", X.device, X.dtype, X.shape)
        _last_dense(dY, "dY")
    dev, shape = X.device, X.shape
    N, C = shape[0], shape[-1]
    P = shape[1] if len(shape) == 3 else 1
    wcode = _CODES[weight.dtype if weight is not None else bias.dtype if bias is not None else _F32]
    L = _lib or lib()
    with _guard(dev, stream):
        if dX is None:
            dX = _like(X)
        if gate is not None and dgate is None:
            dgate = _like(gate)
        dwb = torch.empty((2, C), device=dev, dtype=_F32)
        if strides is not None:
            strides = _longs(*(v for t in (X, dY, gate, dX, dgate) for v in _group_view(t, shape)))
        workspace, nws = _group_work(workspace, N, P, C, groups, 1, dev)
        rc = L.hla2_groupnorm_backward(X.data_ptr(), dY.data_ptr(), stats.data_ptr(), _ptr(weight), _ptr(bias),
                                       _ptr(gate), dX.data_ptr(), _ptr(dgate), dwb.data_ptr(), N, P, C, groups,
                                       strides, acode, _CODES[X.dtype], wcode, _ptr(workspace), nws, _raw(dev, stream))
    if rc:
        _check(rc, "hla2_groupnorm_backward")
    dW, dB = dwb.unbind(0)
    return dX, dW, dB, dgate


def _rotary_checks(Q, pos, freq, sections, K, OQ, OK):
    """The checks of the rotary call, one by one."""
    _operand(Q, "Q")
    if Q.dim() != 4:
        raise ValueError("expected Q [B,H,T,d]")
    _dtype_code(Q)
    B, _, T, _ = Q.shape
    dev = Q.device
    _last_dense(Q, "Q")
    if K is not None:
        _operand(K, "K", dev, Q.dtype)
        if K.dim() != 4 or K.shape[0] != B or K.shape[2:] != Q.shape[2:]:
            raise ValueError("expected K [B,HK,T,d] with Q's B, T and d")
        _last_dense(K, "K")
    elif OK is not None:
        raise ValueError("OK without K")
    axes = len(sections)
    _operand(pos, "pos", dev, torch.int32)
    if pos.shape != (axes, B, T) and pos.shape != (axes, T):
        raise ValueError(f"pos has shape {tuple(pos.shape)}, expected {(axes, B, T)} or {(axes, T)}")
    _last_dense(pos, "pos")
    _operand(freq, "freq", dev, _F32, dense=True)
    if freq.dim() != 1 or sum(sections) != freq.numel():
        raise ValueError(f"freq must hold one frequency for each of the sections' {sum(sections)} pairs")
    if OQ is not None:
        _output(OQ, "OQ", dev, Q.dtype, Q.shape)
    if OK is not None:
        _output(OK, "OK", dev, K.dtype, K.shape)
    _cuda_device(Q, "Q")


def hla2_rotary(Q: torch.Tensor, pos: torch.Tensor, freq: torch.Tensor, sections, K: torch.Tensor | None = None,
                OQ: torch.Tensor | None = None, OK: torch.Tensor | None = None, interleaved: bool = False,
                inverse: bool = False, stream=None):
    """Rotary positions with several axes: pair p of each head's first
    2 * len(freq) channels turns by pos[axis of p] * freq[p] (``inverse``: back,
    which is the gradient).  Q [B,H,T,d], K [B,HK,T,d] fp32 or bf16; pos int32
    [axes,B,T] or [axes,T]; freq fp32 [pairs]; ``sections``: how many pairs
    follow each axis, in order.  Pairs are (p, p + pairs), or (2p, 2p + 1) when
    ``interleaved``.  OQ and OK may be Q and K; those not given take the memory
    order of their input.  Returns (OQ, OK)."""
    sections = tuple(sections)
    shape, dt, dev, axes = Q.shape, Q.dtype, Q.device, len(sections)
    if not (Q.is_cuda and len(shape) == 4 and dt in _CODES and Q.stride(3) == 1 and OQ is None and OK is None and
            pos.dtype is torch.int32 and pos.shape == (axes, shape[0], shape[2]) and pos.is_contiguous() and
            pos.device == dev and freq.dtype is _F32 and freq.shape == (sum(sections),) and freq.is_contiguous() and
            freq.device == dev and
            (K is None or (K.dtype is dt and K.device == dev and K.dim() == 4 and K.stride(3) == 1 and
                           K.shape[0] == shape[0] and K.shape[2:] == shape[2:]))):
        _rotary_checks(Q, pos, freq, sections, K, OQ, OK)
    B, H, T, d = shape
    L = _lib or lib()
    with _guard(dev, stream):
        if OQ is None:
            OQ = _like(Q)
        sq, so, sp = Q.stride(), OQ.stride(), pos.stride()
        pb = sp[1] if len(sp) == 3 else 0
        if K is None:
            HK, pk, po = 0, None, None
            st = _longs(sq[0], sq[1], sq[2], so[0], so[1], so[2], 0, 0, 0, 0, 0, 0, sp[0], pb)
        else:
            if OK is None:
                OK = _like(K)
            HK, pk, po = K.shape[1], K.data_ptr(), OK.data_ptr()
            sk, sl = K.stride(), OK.stride()
            st = _longs(sq[0], sq[1], sq[2], so[0], so[1], so[2], sk[0], sk[1], sk[2], sl[0], sl[1], sl[2], sp[0], pb)
        rc = L.hla2_rotary(Q.data_ptr(), OQ.data_ptr(), pk, po, pos.data_ptr(), freq.data_ptr(), B, H, HK, T, d,
                           2 * freq.numel(), axes, _ints(*sections), bool(interleaved), bool(inverse),
                           st, _CODES[dt], _raw(dev, stream))
    if rc:
        _check(rc, "hla2_rotary")
    return OQ, OK
