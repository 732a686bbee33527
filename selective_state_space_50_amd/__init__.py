"""MI355X (gfx950) selective scan: thin Python binding of libssm.so.

The binding only marshals arguments: it checks tensor dtypes, devices and
contiguity, allocates outputs and the workspace with torch, and passes raw
device pointers plus torch's current HIP stream to the C ABI declared in
``include/ssm.h``.  Every step of the computation runs in the HIP kernels.
There is no CPU fallback: if the library is missing or fails to load, every
call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

__all__ = ["scan_fwd", "scan_fwd_save", "scan_save_sizes", "scan_bwd", "state_update", "scan_plan", "scan_workspace_bytes",
           "scan_bwd_workspace_bytes", "selective_scan", "conv1d_fwd", "conv1d_update", "linattn_fwd", "linattn_bwd",
           "linattn_update", "linattn_workspace_bytes", "linattn_bwd_workspace_bytes", "linear_attention",
           "groupnorm_fwd", "groupnorm_bwd", "groupnorm_workspace_bytes", "group_norm", "rotary_freqs", "rotary_fwd",
           "rotary_bwd", "rotary", "qknorm_fwd", "qknorm_bwd", "qknorm_bwd_workspace_bytes", "qk_norm",
           "ssdconv_fwd", "ssdconv_update", "ssdconv_workspace_bytes", "lib",
           "SSMError", "LIB_PATH",
           "HEADER_PATH", "exported_api"]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssm.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "ssm.h")

SSM_OK, SSM_EINVAL, SSM_EUNSUPPORTED, SSM_EWORKSPACE, SSM_EHIP = range(5)
DTYPE_F32, DTYPE_BF16 = 0, 1
ABI_VERSION = 7     # SSM_ABI_VERSION of include/ssm.h


class SSMError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        self.status = status
        super().__init__(f"{func} failed with status {status} ({_status_name(status)}): {detail}")


class ScanOpts(ctypes.Structure):
    _fields_ = [("chunk_len", ctypes.c_int64), ("states_per_lane", ctypes.c_int32),
                ("time_block", ctypes.c_int32), ("one_block_per_cu", ctypes.c_int32),
                ("a_structure", ctypes.c_int32)]


class Variant(ctypes.Structure):
    _fields_ = [("discretization", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("delta_bias", ctypes.c_void_p)]


DISCRETIZATIONS = {"mamba": 0, "zoh": 1, "bilinear": 2}


class ScanPlan(ctypes.Structure):
    _fields_ = [("chunk_len", ctypes.c_int64), ("n_chunks", ctypes.c_int64),
                ("states_per_lane", ctypes.c_int32), ("waves_per_block", ctypes.c_int32),
                ("time_block", ctypes.c_int32), ("specialised", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_uint64), ("blocks", ctypes.c_uint64),
                ("lds_reserve", ctypes.c_uint64)]


class LinAttnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seqlen", "nheads", "q_heads", "k_heads", "v_heads", "dk", "dv",
                                              "q_row", "k_row", "v_row")] + \
               [("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class RotaryShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "period", "q_heads", "k_heads", "dim", "rot", "q_row", "k_row")] + \
               [("interleaved", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class SsdConvShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "sequences", "max_seqlen", "nheads", "headdim", "dstate", "ngroups",
                                              "width", "nslots", "x_row", "z_row", "delta_row")] + \
               [("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None


def lib():
    """Load libssm.so (built in-tree by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libssm.so not found at {LIB_PATH}: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    # torch first: its HIP runtime is then the one libssm.so binds to (a process must not
    # load a second copy of the runtime, which would see no devices)
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    L = ctypes.CDLL(LIB_PATH)
    I64, I32, P, SZ = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    L.ssm_abi_version.restype = I32
    L.ssm_abi_version.argtypes = []
    L.ssm_status_str.restype = ctypes.c_char_p
    L.ssm_status_str.argtypes = [I32]
    L.ssm_last_error.restype = ctypes.c_char_p
    L.ssm_last_error.argtypes = []
    L.ssm_scan_plan_get.restype = I32
    L.ssm_scan_plan_get.argtypes = [I64, I64, I64, I64, I32, ctypes.POINTER(ScanOpts),
                                    ctypes.POINTER(ScanPlan)]
    L.ssm_scan_workspace_bytes.restype = SZ
    L.ssm_scan_workspace_bytes.argtypes = [I64, I64, I64, I64, I32, ctypes.POINTER(ScanOpts)]
    L.ssm_scan_fwd.restype = I32
    L.ssm_scan_fwd.argtypes = [I64, I64, I64, I64, I32, P, P, P, P, P, P, P, P, P, P, I32,
                               ctypes.POINTER(Variant), ctypes.POINTER(ScanOpts), P, SZ, P]
    L.ssm_issue_probe.restype = I32
    L.ssm_issue_probe.argtypes = [I32, I64, I64, I64, P, P]
    L.ssm_noalloc_scratch_bytes.restype = SZ
    L.ssm_noalloc_scratch_bytes.argtypes = []
    L.ssm_scan_fwd_noalloc.restype = I32
    L.ssm_scan_fwd_noalloc.argtypes = [I64, I64, I64, I64, I32, P, P, P, P, P, P, P, P, P, P, I32,
                                       ctypes.POINTER(Variant), ctypes.POINTER(ScanOpts), P]
    L.ssm_state_update.restype = I32
    L.ssm_state_update.argtypes = [I64, I64, I64, I32, P, P, P, P, P, P, P, P, P, I32,
                                   ctypes.POINTER(Variant), P]
    L.ssm_scan_bwd_workspace_bytes.restype = SZ
    L.ssm_scan_bwd_workspace_bytes.argtypes = [I64, I64, I64, I64, I32, I32]
    L.ssm_scan_bwd.restype = I32
    L.ssm_scan_bwd.argtypes = [I64, I64, I64, I64, I32] + [P] * 18 + [I32, I32, P, P, P, P, SZ, P]
    L.ssm_scan_save_sizes.restype = I32
    L.ssm_scan_save_sizes.argtypes = [I64, I64, I64, I64, I32, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
    L.ssm_scan_fwd_save.restype = I32
    L.ssm_scan_fwd_save.argtypes = [I64, I64, I64, I64, I32] + [P] * 10 + [I32, ctypes.POINTER(Variant), P, P, SZ, P]
    L.ssm_conv1d_fwd.restype = I32
    L.ssm_conv1d_fwd.argtypes = [I64, I64, I64, I64, I32, P, P, P, P, P, P, I32, P]
    L.ssm_ssd_fwd.restype = I32
    L.ssm_ssd_fwd.argtypes = [I64, I64, I64, I64, I64, I64, I32] + [P] * 11 + [I32, P]
    L.ssm_ssd_bwd_workspace_bytes.restype = SZ
    L.ssm_ssd_bwd_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I32]
    L.ssm_ssd_bwd.restype = I32
    L.ssm_ssd_bwd.argtypes = [I64, I64, I64, I64, I64, I64, I32] + [P] * 20 + [I32, P, SZ, P]
    L.ssm_conv1d_update.restype = I32
    L.ssm_conv1d_update.argtypes = [I64, I64, I64, I32, P, P, P, P, P, I32, P]
    L.ssm_conv1d_bwd_workspace_bytes.restype = SZ
    L.ssm_conv1d_bwd_workspace_bytes.argtypes = [I64, I64, I64, I64, I32]
    L.ssm_conv1d_bwd.restype = I32
    L.ssm_conv1d_bwd.argtypes = [I64, I64, I64, I64, I32] + [P] * 9 + [I32, P, SZ, P]
    S = ctypes.POINTER(LinAttnShape)
    L.ssm_linattn_workspace_bytes.restype = SZ
    L.ssm_linattn_workspace_bytes.argtypes = [S]
    L.ssm_linattn_fwd.restype = I32
    L.ssm_linattn_fwd.argtypes = [S, P, P, P, P, ctypes.c_float, P, P, P, P, P, SZ, P]
    L.ssm_linattn_bwd_workspace_bytes.restype = SZ
    L.ssm_linattn_bwd_workspace_bytes.argtypes = [S, I32]
    L.ssm_linattn_bwd.restype = I32
    L.ssm_linattn_bwd.argtypes = [S, P, P, P, P, ctypes.c_float] + [P] * 10 + [SZ, P]
    L.ssm_linattn_update.restype = I32
    L.ssm_linattn_update.argtypes = [S, P, P, P, P, P, ctypes.c_float, P, P]
    L.ssm_groupnorm_workspace_bytes.restype = SZ
    L.ssm_groupnorm_workspace_bytes.argtypes = [I64, I64, I64, I64, I32, I32]
    L.ssm_groupnorm_fwd.restype = I32
    L.ssm_groupnorm_fwd.argtypes = [I64, I64, I64, I64, I32, P, P, P, P, ctypes.c_float, I32, P, P, P, P, SZ, P]
    L.ssm_groupnorm_bwd.restype = I32
    L.ssm_groupnorm_bwd.argtypes = [I64, I64, I64, I64, I32, P, P, P, P, I32] + [P] * 8 + [SZ, P]
    R, F = ctypes.POINTER(RotaryShape), ctypes.c_float
    L.ssm_rotary_fwd.restype = I32
    L.ssm_rotary_fwd.argtypes = [R, P, P, P, P, F, I32, P, P, P]
    L.ssm_qknorm_fwd.restype = I32
    L.ssm_qknorm_fwd.argtypes = [R] + [P] * 6 + [F, F, P, P, P]
    L.ssm_qknorm_bwd_workspace_bytes.restype = SZ
    L.ssm_qknorm_bwd_workspace_bytes.argtypes = [R]
    L.ssm_qknorm_bwd.restype = I32
    L.ssm_qknorm_bwd.argtypes = [R] + [P] * 6 + [F, F] + [P] * 7 + [SZ, P]
    C = ctypes.POINTER(SsdConvShape)
    for f in (L.ssm_ssdconv_workspace_bytes, L.ssm_ssdconv_update_workspace_bytes):
        f.restype, f.argtypes = SZ, [C]
    L.ssm_ssdconv_fwd.restype = I32
    L.ssm_ssdconv_fwd.argtypes = [C] + [P] * 8 + [I32] + [P] * 7 + [SZ, P]
    L.ssm_ssdconv_update.restype = I32
    L.ssm_ssdconv_update.argtypes = [C] + [P] * 8 + [I32] + [P] * 5 + [SZ, P]
    if L.ssm_abi_version() != ABI_VERSION:
        raise ImportError(f"libssm ABI version {L.ssm_abi_version()} != {ABI_VERSION}")
    _lib = L
    return L


def _status_name(status: int) -> str:
    try:
        return lib().ssm_status_str(status).decode()
    except Exception:  # pragma: no cover - used while building an error message
        return "?"


def _check(status: int, func: str):
    if status != SSM_OK:
        raise SSMError(status, func, lib().ssm_last_error().decode())


def exported_api():
    """Function names declared in include/ssm.h."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(ssm_[a-z_]+)\s*\(", text)))


def _opts(chunk_len=0, states_per_lane=0, time_block=0, one_block_per_cu=0, general_a=False):
    if not (chunk_len or states_per_lane or time_block or one_block_per_cu or general_a):
        return None
    return ScanOpts(int(chunk_len), int(states_per_lane), int(time_block), int(one_block_per_cu),
                    -1 if general_a else 0)


def _variant(discretization, delta_bias, dim, device):
    """The ssm_variant of a call (None for the default: Mamba, no delta bias)."""
    import torch
    if discretization not in DISCRETIZATIONS:
        raise ValueError(f"discretization {discretization!r} is not one of {sorted(DISCRETIZATIONS)}")
    _need(delta_bias, "delta_bias", (dim,), torch.float32, device)
    if discretization == "mamba" and delta_bias is None:
        return None
    return Variant(DISCRETIZATIONS[discretization], 0, _ptr(delta_bias))


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def scan_plan(batch, seqlen, dim, dstate, dtype="bf16", chunk_len=0, states_per_lane=0,
              time_block=0, one_block_per_cu=0) -> dict:
    """What ssm_scan_fwd will launch for this shape (host-only)."""
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    p = ScanPlan()
    o = _opts(chunk_len, states_per_lane, time_block, one_block_per_cu)
    _check(lib().ssm_scan_plan_get(batch, seqlen, dim, dstate, code,
                                   ctypes.byref(o) if o else None, ctypes.byref(p)),
           "ssm_scan_plan_get")
    return {k: getattr(p, k) for k, _ in ScanPlan._fields_}


def scan_workspace_bytes(batch, seqlen, dim, dstate, dtype="bf16", chunk_len=0,
                         states_per_lane=0, time_block=0, one_block_per_cu=0) -> int:
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    o = _opts(chunk_len, states_per_lane, time_block, one_block_per_cu)
    return int(lib().ssm_scan_workspace_bytes(batch, seqlen, dim, dstate, code,
                                              ctypes.byref(o) if o else None))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, shape, dtype, device):
    if t is None or (t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous()):
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _aligned(t):
    """t, or a copy where t does not start on 16 bytes (a part of another tensor may not), as the library needs it."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _gradient(g):
    """An incoming gradient as the library takes one: contiguous and on 16 bytes (torch's cat, for one, hands out
    parts of a larger gradient)."""
    return None if g is None else _aligned(g.contiguous())


def _workspace(given, need, device):
    """The caller's workspace where it is large enough, else a new one.  (A kernel writes ``need`` bytes from its
    address on: it has to lie in one piece on the tensors' device.)"""
    import torch
    if given is not None and given.device != device:
        raise ValueError(f"workspace is on {given.device}, expected {device}")
    if given is not None and not given.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if need and (given is None or given.numel() * given.element_size() < need):
        return torch.empty(need, dtype=torch.uint8, device=device)
    return given


def _written(*tensors):
    """Tell autograd that the library writes these (its pointers do not): a backward that has saved one of them then
    raises, as after torch's own in-place operations."""
    import torch
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def scan_fwd(x, delta, A, B, C, D=None, z=None, h0=None, *, delta_softplus=False,
             discretization="mamba", delta_bias=None,
             return_last_state=False, out=None, h_last=None, workspace=None, chunk_len=0,
             states_per_lane=0, time_block=0, one_block_per_cu=0, general_a=False, stream=None):
    """Selective scan y = S6(x, delta, A, B, C, D) [* silu(z)] on the GPU.

    x, delta, z: [B, L, D];  B, C: [B, L, N];  A: [D, N] fp32;  D: [D] fp32;
    h0: [B, D, N] fp32.  x/delta/z/B/C share one dtype (bfloat16 or float32).
    discretization: "mamba" (A_bar = exp(dt A), B_bar = dt B), "zoh" or "bilinear";
    delta_bias: [D] fp32 added to delta before the softplus.
    general_a: always one exp per state (never the structured-A path, ssm_scan_opts.a_structure).
    Returns y (same dtype as x), or (y, h_last) when return_last_state.
    """
    import torch
    if x.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be [batch, seqlen, dim] and A [dim, dstate]")
    Bsz, L, Dm = x.shape
    N = A.shape[1]
    dev, dt = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("scan_fwd runs on the GPU only; tensors must be on a cuda device")
    _need(x, "x", (Bsz, L, Dm), dt, dev)
    _need(delta, "delta", (Bsz, L, Dm), dt, dev)
    _need(z, "z", (Bsz, L, Dm), dt, dev)
    _need(B, "B", (Bsz, L, N), dt, dev)
    _need(C, "C", (Bsz, L, N), dt, dev)
    _need(A, "A", (Dm, N), torch.float32, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    _need(h0, "h0", (Bsz, Dm, N), torch.float32, dev)
    v = _variant(discretization, delta_bias, Dm, dev)
    code = _dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", (Bsz, L, Dm), dt, dev)
    if return_last_state and h_last is None:
        h_last = torch.empty((Bsz, Dm, N), dtype=torch.float32, device=dev)
    _need(h_last, "h_last", (Bsz, Dm, N), torch.float32, dev)
    o = _opts(chunk_len, states_per_lane, time_block, one_block_per_cu, general_a)
    ws_bytes = int(lib().ssm_scan_workspace_bytes(Bsz, L, Dm, N, code, ctypes.byref(o) if o else None))
    workspace = _workspace(workspace, ws_bytes, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    st = lib().ssm_scan_fwd(Bsz, L, Dm, N, code, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
                            _ptr(D), _ptr(z), _ptr(h0), _ptr(h_last), _ptr(out),
                            int(bool(delta_softplus)), ctypes.byref(v) if v else None,
                            ctypes.byref(o) if o else None,
                            _ptr(workspace) if ws_bytes else None, ws_bytes,
                            ctypes.c_void_p(s.cuda_stream))
    _check(st, "ssm_scan_fwd")
    _written(out, h_last)
    return (out, h_last) if return_last_state else out


def scan_fwd_noalloc(x, delta, A, B, C, D=None, z=None, h0=None, *, delta_softplus=False,
                     discretization="mamba", delta_bias=None, out=None, h_last=None, chunk_len=0,
                     states_per_lane=0, general_a=False, stream=None):
    """scan_fwd through ssm_scan_fwd_noalloc: the library's fixed scratch array stands in for
    the workspace, so the call itself allocates no device memory when ``out`` (and
    ``h_last``, if wanted) are given.  Returns y, or (y, h_last) when h_last is given."""
    import torch
    if x.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be [batch, seqlen, dim] and A [dim, dstate]")
    Bsz, L, Dm = x.shape
    N = A.shape[1]
    dev, dt = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("scan_fwd_noalloc runs on the GPU only; tensors must be on a cuda device")
    for t, name, shape, tdt in ((x, "x", (Bsz, L, Dm), dt), (delta, "delta", (Bsz, L, Dm), dt),
                                (z, "z", (Bsz, L, Dm), dt), (B, "B", (Bsz, L, N), dt),
                                (C, "C", (Bsz, L, N), dt), (A, "A", (Dm, N), torch.float32),
                                (D, "D", (Dm,), torch.float32), (h0, "h0", (Bsz, Dm, N), torch.float32),
                                (h_last, "h_last", (Bsz, Dm, N), torch.float32)):
        _need(t, name, shape, tdt, dev)
    v = _variant(discretization, delta_bias, Dm, dev)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", (Bsz, L, Dm), dt, dev)
    o = _opts(chunk_len, states_per_lane, 0, 0, general_a)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    st = lib().ssm_scan_fwd_noalloc(Bsz, L, Dm, N, _dtype_code(x), _ptr(x), _ptr(delta), _ptr(A), _ptr(B),
                                    _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(h_last), _ptr(out),
                                    int(bool(delta_softplus)), ctypes.byref(v) if v else None,
                                    ctypes.byref(o) if o else None, ctypes.c_void_p(s.cuda_stream))
    _check(st, "ssm_scan_fwd_noalloc")
    _written(out, h_last)
    return (out, h_last) if h_last is not None else out


def issue_rates(workgroups=256, waves_per_workgroup=16, iters=4096, reps=5):
    """Measured VALU issue rates (lane operations per second) of an fp32 FMA, v_exp_f32 and
    v_rcp_f32 on the current GPU (ssm_issue_probe, timed with events; median of reps)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device())
    sink = torch.empty(64 * waves_per_workgroup, dtype=torch.float32, device=dev)
    s = torch.cuda.current_stream(dev)
    ops = workgroups * waves_per_workgroup * 64 * 8 * iters
    out = {}
    for op, name in ((0, "fma"), (1, "exp"), (2, "rcp")):
        times = []
        for r in range(reps + 1):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record(s)
            _check(lib().ssm_issue_probe(op, workgroups, waves_per_workgroup, iters, _ptr(sink),
                                         ctypes.c_void_p(s.cuda_stream)), "ssm_issue_probe")
            e1.record(s)
            e1.synchronize()
            if r:
                times.append(e0.elapsed_time(e1))
        times.sort()
        out[name] = ops / (times[len(times) // 2] * 1e-3)
    return out


def state_update(h, x, delta, A, B, C, D=None, z=None, *, delta_softplus=False,
                 discretization="mamba", delta_bias=None, out=None, stream=None):
    """One recurrent step: updates h [B, D, N] fp32 in place and returns y [B, D].

    x, delta, z: [B, D];  B, C: [B, N];  A: [D, N] fp32;  D: [D] fp32;
    discretization and delta_bias as for scan_fwd.
    """
    import torch
    if h.dim() != 3:
        raise ValueError("h must be [batch, dim, dstate]")
    Bsz, Dm, N = h.shape
    dev, dt = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("state_update runs on the GPU only; tensors must be on a cuda device")
    _need(h, "h", (Bsz, Dm, N), torch.float32, dev)
    _need(x, "x", (Bsz, Dm), dt, dev)
    _need(delta, "delta", (Bsz, Dm), dt, dev)
    _need(z, "z", (Bsz, Dm), dt, dev)
    _need(B, "B", (Bsz, N), dt, dev)
    _need(C, "C", (Bsz, N), dt, dev)
    _need(A, "A", (Dm, N), torch.float32, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    v = _variant(discretization, delta_bias, Dm, dev)
    code = _dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", (Bsz, Dm), dt, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    st = lib().ssm_state_update(Bsz, Dm, N, code, _ptr(h), _ptr(x), _ptr(delta), _ptr(A), _ptr(B),
                                _ptr(C), _ptr(D), _ptr(z), _ptr(out), int(bool(delta_softplus)),
                                ctypes.byref(v) if v else None, ctypes.c_void_p(s.cuda_stream))
    _check(st, "ssm_state_update")
    _written(h, out)
    return out


def scan_bwd_workspace_bytes(batch, seqlen, dim, dstate, dtype="bf16", saved_checkpoints=False) -> int:
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    return int(lib().ssm_scan_bwd_workspace_bytes(batch, seqlen, dim, dstate, code, int(bool(saved_checkpoints))))


def scan_save_sizes(batch, seqlen, dim, dstate, dtype="bf16"):
    """(workspace bytes, checkpoint bytes) of scan_fwd_save at this shape."""
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    ws, ck = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().ssm_scan_save_sizes(batch, seqlen, dim, dstate, code, ctypes.byref(ws), ctypes.byref(ck)),
           "ssm_scan_save_sizes")
    return int(ws.value), int(ck.value)


def scan_fwd_save(x, delta, A, B, C, D=None, z=None, h0=None, *, delta_softplus=False,
                  discretization="mamba", delta_bias=None, return_last_state=False, out=None,
                  h_last=None, checkpoints=None, workspace=None, stream=None):
    """scan_fwd that also stores the state before every 8th step for scan_bwd (its
    ``checkpoints`` argument), on the backward's sequence chunking.  Arguments as
    scan_fwd (dstate 16 and dim a multiple of 64 only).  Returns (y, checkpoints), or
    (y, h_last, checkpoints) when return_last_state; checkpoints is a flat fp32 tensor
    [B, ceil(L/8), N, D]."""
    import torch
    if x.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be [batch, seqlen, dim] and A [dim, dstate]")
    Bsz, L, Dm = x.shape
    N = A.shape[1]
    dev, dt = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("scan_fwd_save runs on the GPU only; tensors must be on a cuda device")
    for t, name, shape, tdt in ((x, "x", (Bsz, L, Dm), dt), (delta, "delta", (Bsz, L, Dm), dt),
                                (z, "z", (Bsz, L, Dm), dt), (B, "B", (Bsz, L, N), dt), (C, "C", (Bsz, L, N), dt),
                                (A, "A", (Dm, N), torch.float32), (D, "D", (Dm,), torch.float32),
                                (h0, "h0", (Bsz, Dm, N), torch.float32)):
        _need(t, name, shape, tdt, dev)
    v = _variant(discretization, delta_bias, Dm, dev)
    code = _dtype_code(x)
    ws_bytes, ck_bytes = scan_save_sizes(Bsz, L, Dm, N, "bf16" if code == DTYPE_BF16 else "f32")
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", (Bsz, L, Dm), dt, dev)
    if return_last_state and h_last is None:
        h_last = torch.empty((Bsz, Dm, N), dtype=torch.float32, device=dev)
    _need(h_last, "h_last", (Bsz, Dm, N), torch.float32, dev)
    nck = (L + 7) // 8
    if checkpoints is None:
        checkpoints = torch.empty((Bsz, nck, N, Dm), dtype=torch.float32, device=dev)
    _need(checkpoints, "checkpoints", (Bsz, nck, N, Dm), torch.float32, dev)
    if not checkpoints.is_contiguous() or checkpoints.numel() * 4 != ck_bytes:
        raise ValueError(f"checkpoints must be a contiguous fp32 tensor of {ck_bytes} bytes")
    workspace = _workspace(workspace, ws_bytes, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    st = lib().ssm_scan_fwd_save(Bsz, L, Dm, N, code, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
                                 _ptr(D), _ptr(z), _ptr(h0), _ptr(h_last), _ptr(out),
                                 int(bool(delta_softplus)), ctypes.byref(v) if v else None,
                                 _ptr(checkpoints), _ptr(workspace) if ws_bytes else None, ws_bytes,
                                 ctypes.c_void_p(s.cuda_stream))
    _check(st, "ssm_scan_fwd_save")
    _written(out, h_last, checkpoints)
    return (out, h_last, checkpoints) if return_last_state else (out, checkpoints)


def scan_bwd(x, delta, A, B, C, D=None, z=None, h0=None, dy=None, dh_last=None, *,
             delta_softplus=False, discretization="mamba", delta_bias=None, need_dh0=True,
             checkpoints=None, workspace=None, stream=None):
    """Gradients of a loss through scan_fwd, given dy = dLoss/dy [B, L, D] (same dtype as
    x) and optionally dh_last = dLoss/dh_last [B, D, N] fp32.  discretization and
    delta_bias [D] fp32: as in scan_fwd.  checkpoints: what scan_fwd_save stored for these
    same inputs (the call then skips its own forward sweep), or None.

    Returns a dict: dx, ddelta, dz (None without z) in x's dtype [B, L, D]; dB, dC in
    x's dtype [B, L, N]; dA [D, N], dD [D] (None without D), ddelta_bias [D] (None
    without a bias) and dh0 [B, D, N] in fp32 (dh0 None when need_dh0 is false).
    """
    import torch
    if x.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be [batch, seqlen, dim] and A [dim, dstate]")
    Bsz, L, Dm = x.shape
    N = A.shape[1]
    dev, dt = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("scan_bwd runs on the GPU only; tensors must be on a cuda device")
    if dy is None:
        raise ValueError("dy is required")
    if discretization not in DISCRETIZATIONS:
        raise ValueError(f"discretization {discretization!r} is not one of {sorted(DISCRETIZATIONS)}")
    for t, name, shape, tdt in ((x, "x", (Bsz, L, Dm), dt), (delta, "delta", (Bsz, L, Dm), dt),
                                (z, "z", (Bsz, L, Dm), dt), (B, "B", (Bsz, L, N), dt),
                                (C, "C", (Bsz, L, N), dt), (A, "A", (Dm, N), torch.float32),
                                (D, "D", (Dm,), torch.float32), (h0, "h0", (Bsz, Dm, N), torch.float32),
                                (dy, "dy", (Bsz, L, Dm), dt), (dh_last, "dh_last", (Bsz, Dm, N), torch.float32),
                                (delta_bias, "delta_bias", (Dm,), torch.float32)):
        _need(t, name, shape, tdt, dev)
    if checkpoints is not None:
        _need(checkpoints, "checkpoints", (Bsz, (L + 7) // 8, N, Dm), torch.float32, dev)
    code = _dtype_code(x)
    out = {"dx": torch.empty_like(x), "ddelta": torch.empty_like(x),
           "dz": torch.empty_like(x) if z is not None else None,
           "dB": torch.empty((Bsz, L, N), dtype=dt, device=dev),
           "dC": torch.empty((Bsz, L, N), dtype=dt, device=dev),
           "dA": torch.empty((Dm, N), dtype=torch.float32, device=dev),
           "dD": torch.empty((Dm,), dtype=torch.float32, device=dev) if D is not None else None,
           "dh0": torch.empty((Bsz, Dm, N), dtype=torch.float32, device=dev) if need_dh0 else None,
           "ddelta_bias": torch.empty((Dm,), dtype=torch.float32, device=dev) if delta_bias is not None else None}
    ws_bytes = int(lib().ssm_scan_bwd_workspace_bytes(Bsz, L, Dm, N, code, int(checkpoints is not None)))
    workspace = _workspace(workspace, ws_bytes, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    st = lib().ssm_scan_bwd(Bsz, L, Dm, N, code, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
                            _ptr(D), _ptr(z), _ptr(h0), _ptr(dy), _ptr(dh_last), _ptr(out["dx"]),
                            _ptr(out["ddelta"]), _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]),
                            _ptr(out["dD"]), _ptr(out["dz"]), _ptr(out["dh0"]), int(bool(delta_softplus)),
                            DISCRETIZATIONS[discretization], _ptr(delta_bias), _ptr(out["ddelta_bias"]),
                            _ptr(checkpoints), _ptr(workspace) if ws_bytes else None, ws_bytes,
                            ctypes.c_void_p(s.cuda_stream))
    _check(st, "ssm_scan_bwd")
    return out


def selective_scan(x, delta, A, B, C, D=None, z=None, h0=None, delta_softplus=False, delta_bias=None,
                   discretization="mamba"):
    """Differentiable selective scan: y = scan_fwd(...) with a torch autograd backward
    through scan_bwd (gradients for every tensor argument, delta_bias included).  The
    forward stores the state checkpoints (scan_fwd_save) when the shape allows them
    (dstate 16, dim a multiple of 64), so that the backward skips its own forward
    sweep."""
    import torch

    class _Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, delta, A, B, C, D, z, h0, delta_bias):
            ck = None
            if A.shape[1] == 16 and x.shape[2] % 64 == 0 and x.shape[1] > 0:
                y, ck = scan_fwd_save(x, delta, A, B, C, D, z, h0, delta_softplus=delta_softplus,
                                      discretization=discretization, delta_bias=delta_bias)
            else:
                y = scan_fwd(x, delta, A, B, C, D, z, h0, delta_softplus=delta_softplus,
                             discretization=discretization, delta_bias=delta_bias)
            ctx.save_for_backward(x, delta, A, B, C, D, z, h0, delta_bias, ck)
            return y

        @staticmethod
        def backward(ctx, gy):
            x, delta, A, B, C, D, z, h0, delta_bias, ck = ctx.saved_tensors
            g = scan_bwd(x, delta, A, B, C, D, z, h0, _gradient(gy), delta_softplus=delta_softplus,
                         discretization=discretization, delta_bias=delta_bias, checkpoints=ck, need_dh0=h0 is not None and ctx.needs_input_grad[7])
            return (g["dx"], g["ddelta"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["dh0"],
                    g["ddelta_bias"])

    return _Scan.apply(x, delta, A, B, C, D, z, h0, delta_bias)


def conv1d_fwd(x, w, bias=None, state=None, *, silu=True, return_state=False, out=None, stream=None):
    """Causal depthwise convolution along the sequence (+ SiLU): x [B, L, D] (bf16 or
    fp32), w [D, W] fp32 (W <= 4), bias [D] fp32, state [B, D, W-1] in x's dtype (the
    inputs before the sequence).  Returns y (and the final state when return_state)."""
    import torch
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must be [batch, seqlen, dim] and w [dim, width]")
    Bsz, L, Dm = x.shape
    W = w.shape[1]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("conv1d_fwd runs on the GPU only; tensors must be on a cuda device")
    _need(w, "w", (Dm, W), torch.float32, dev)
    _need(bias, "bias", (Dm,), torch.float32, dev)
    _need(state, "state", (Bsz, Dm, W - 1), x.dtype, dev)
    _need(x, "x", (Bsz, L, Dm), x.dtype, dev)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", (Bsz, L, Dm), x.dtype, dev)
    st_out = torch.empty((Bsz, Dm, W - 1), dtype=x.dtype, device=dev) if return_state else None
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    _check(lib().ssm_conv1d_fwd(Bsz, L, Dm, W, _dtype_code(x), _ptr(x), _ptr(w), _ptr(bias), _ptr(state),
                                _ptr(out), _ptr(st_out), int(bool(silu)), ctypes.c_void_p(s.cuda_stream)),
           "ssm_conv1d_fwd")
    _written(out)
    return (out, st_out) if return_state else out


def conv1d_bwd_workspace_bytes(batch, seqlen, dim, width, dtype="bf16") -> int:
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    return int(lib().ssm_conv1d_bwd_workspace_bytes(batch, seqlen, dim, width, code))


def conv1d_bwd(x, w, bias=None, state=None, dy=None, *, silu=True, need_dstate=None, workspace=None, stream=None):
    """Gradients of a loss through conv1d_fwd given dy = dLoss/dy [B, L, D] (x's dtype).
    Returns a dict: dx [B, L, D] (x's dtype), dw [D, W] fp32, dbias [D] fp32 (None without
    a bias) and dstate [B, D, W-1] (x's dtype; by default only when a state is given)."""
    import torch
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must be [batch, seqlen, dim] and w [dim, width]")
    Bsz, L, Dm = x.shape
    W = w.shape[1]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("conv1d_bwd runs on the GPU only; tensors must be on a cuda device")
    if dy is None:
        raise ValueError("dy is required")
    _need(w, "w", (Dm, W), torch.float32, dev)
    _need(bias, "bias", (Dm,), torch.float32, dev)
    _need(state, "state", (Bsz, Dm, W - 1), x.dtype, dev)
    _need(x, "x", (Bsz, L, Dm), x.dtype, dev)
    _need(dy, "dy", (Bsz, L, Dm), x.dtype, dev)
    if need_dstate is None:
        need_dstate = state is not None
    out = {"dx": torch.empty_like(x), "dw": torch.empty((Dm, W), dtype=torch.float32, device=dev),
           "dbias": torch.empty((Dm,), dtype=torch.float32, device=dev) if bias is not None else None,
           "dstate": torch.empty((Bsz, Dm, W - 1), dtype=x.dtype, device=dev) if need_dstate else None}
    code = _dtype_code(x)
    ws_bytes = int(lib().ssm_conv1d_bwd_workspace_bytes(Bsz, L, Dm, W, code))
    workspace = _workspace(workspace, ws_bytes, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    _check(lib().ssm_conv1d_bwd(Bsz, L, Dm, W, code, _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(dy),
                                _ptr(out["dx"]), _ptr(out["dw"]), _ptr(out["dbias"]), _ptr(out["dstate"]),
                                int(bool(silu)), _ptr(workspace) if ws_bytes else None, ws_bytes,
                                ctypes.c_void_p(s.cuda_stream)), "ssm_conv1d_bwd")
    return out


def causal_conv1d(x, w, bias=None, state=None, silu=True):
    """Differentiable causal depthwise convolution (+ SiLU): y = conv1d_fwd(...) with a
    torch autograd backward through conv1d_bwd (gradients for x, w, bias and state)."""
    import torch

    class _Conv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, bias, state):
            y = conv1d_fwd(x, w, bias, state, silu=silu)
            ctx.save_for_backward(x, w, bias, state)
            return y

        @staticmethod
        def backward(ctx, gy):
            x, w, bias, state = ctx.saved_tensors
            g = conv1d_bwd(x, w, bias, state, _gradient(gy), silu=silu,
                           need_dstate=state is not None and ctx.needs_input_grad[3])
            return g["dx"], g["dw"], g["dbias"], g["dstate"]

    return _Conv.apply(x, w, bias, state)


def conv1d_update(state, x, w, bias=None, *, silu=True, out=None, stream=None):
    """One token of conv1d_fwd: state [B, D, W-1] (x's dtype) updated in place, x [B, D];
    returns y [B, D]."""
    import torch
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [batch, dim] and w [dim, width]")
    Bsz, Dm = x.shape
    W = w.shape[1]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("conv1d_update runs on the GPU only; tensors must be on a cuda device")
    _need(w, "w", (Dm, W), torch.float32, dev)
    _need(bias, "bias", (Dm,), torch.float32, dev)
    _need(state, "state", (Bsz, Dm, W - 1), x.dtype, dev)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", (Bsz, Dm), x.dtype, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    _check(lib().ssm_conv1d_update(Bsz, Dm, W, _dtype_code(x), _ptr(state), _ptr(x), _ptr(w), _ptr(bias),
                                   _ptr(out), int(bool(silu)), ctypes.c_void_p(s.cuda_stream)),
           "ssm_conv1d_update")
    _written(state, out)
    return out


def ssd_fwd(x, delta, A, B, C, D=None, z=None, h0=None, *, delta_softplus=False, delta_bias=None,
            return_last_state=False, out=None, h_last=None, stream=None):
    """Multi-head SSD scan (the Mamba-2 layer's state space model) on the GPU.

    x, z: [B, L, H, P];  delta: [B, L, H];  B, C: [B, L, N], or [B, L, G, N] for G groups
    of H / G consecutive heads each sharing one B and C row (all bf16, or all fp32);
    A, D, delta_bias: [H] fp32;  h0: [B, H, P, N] fp32.  P = 64, N = 128 in bf16 runs on the
    matrix cores; other P, N <= 256 and fp32 on the generic scan kernel.  Returns y
    [B, L, H, P] (x's dtype), or (y, h_last) when return_last_state.
    """
    import torch
    if x.dim() != 4 or A.dim() != 1:
        raise ValueError("x must be [batch, seqlen, nheads, headdim] and A [nheads]")
    Bsz, L, H, P = x.shape
    N = B.shape[-1]
    G = B.shape[2] if B.dim() == 4 else 1
    bc_shape = (Bsz, L, G, N) if B.dim() == 4 else (Bsz, L, N)
    dev, dt = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("ssd_fwd runs on the GPU only; tensors must be on a cuda device")
    _need(delta, "delta", (Bsz, L, H), dt, dev)
    _need(z, "z", (Bsz, L, H, P), dt, dev)
    _need(B, "B", bc_shape, dt, dev)
    _need(C, "C", bc_shape, dt, dev)
    _need(A, "A", (H,), torch.float32, dev)
    _need(D, "D", (H,), torch.float32, dev)
    _need(delta_bias, "delta_bias", (H,), torch.float32, dev)
    _need(h0, "h0", (Bsz, H, P, N), torch.float32, dev)
    code = _dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", (Bsz, L, H, P), dt, dev)
    if return_last_state and h_last is None:
        h_last = torch.empty((Bsz, H, P, N), dtype=torch.float32, device=dev)
    _need(h_last, "h_last", (Bsz, H, P, N), torch.float32, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    st = lib().ssm_ssd_fwd(Bsz, L, H, P, N, G, code, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                           _ptr(z), _ptr(delta_bias), _ptr(h0), _ptr(h_last), _ptr(out),
                           int(bool(delta_softplus)), ctypes.c_void_p(s.cuda_stream))
    _check(st, "ssm_ssd_fwd")
    _written(out, h_last)
    return (out, h_last) if return_last_state else out


def ssd_bwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, dtype="bf16") -> int:
    """Device workspace bytes of ssd_bwd for this shape (0: nothing to compute)."""
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    return int(lib().ssm_ssd_bwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, code))


def ssd_bwd(x, delta, A, B, C, D=None, z=None, h0=None, dy=None, dh_last=None, *, delta_softplus=False,
            delta_bias=None, workspace=None, stream=None):
    """Gradients of a loss through ssd_fwd (one B/C group: B, C [B, L, N]), given dy =
    dLoss/dy [B, L, H, P] (x's dtype) and optionally dh_last = dLoss/dh_last [B, H, P, N] fp32.

    Returns a dict: dx, dz (None without z) [B, L, H, P] and ddelta [B, L, H] and dB, dC
    [B, L, N] in x's dtype; dA, dD (None without D), ddelta_bias (None without a bias) [H] and
    dh0 [B, H, P, N] in fp32.
    """
    import torch
    if x.dim() != 4 or A.dim() != 1:
        raise ValueError("x must be [batch, seqlen, nheads, headdim] and A [nheads]")
    if B.dim() != 3:
        raise ValueError("ssd_bwd takes one B/C group: B and C [batch, seqlen, dstate]")
    Bsz, L, H, P = x.shape
    N = B.shape[-1]
    dev, dt = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("ssd_bwd runs on the GPU only; tensors must be on a cuda device")
    if dy is None:
        raise ValueError("dy is required")
    for t, name, shape, tdt in ((delta, "delta", (Bsz, L, H), dt), (z, "z", (Bsz, L, H, P), dt),
                                (B, "B", (Bsz, L, N), dt), (C, "C", (Bsz, L, N), dt), (A, "A", (H,), torch.float32),
                                (D, "D", (H,), torch.float32), (delta_bias, "delta_bias", (H,), torch.float32),
                                (h0, "h0", (Bsz, H, P, N), torch.float32), (dy, "dy", (Bsz, L, H, P), dt),
                                (dh_last, "dh_last", (Bsz, H, P, N), torch.float32)):
        _need(t, name, shape, tdt, dev)
    code = _dtype_code(x)
    f32 = torch.float32
    out = {"dx": torch.empty_like(x), "ddelta": torch.empty((Bsz, L, H), dtype=dt, device=dev),
           "dz": torch.empty_like(x) if z is not None else None,
           "dB": torch.empty((Bsz, L, N), dtype=dt, device=dev), "dC": torch.empty((Bsz, L, N), dtype=dt, device=dev),
           "dA": torch.empty((H,), dtype=f32, device=dev),
           "dD": torch.empty((H,), dtype=f32, device=dev) if D is not None else None,
           "ddelta_bias": torch.empty((H,), dtype=f32, device=dev) if delta_bias is not None else None,
           "dh0": torch.empty((Bsz, H, P, N), dtype=f32, device=dev)}
    ws_bytes = int(lib().ssm_ssd_bwd_workspace_bytes(Bsz, L, H, P, N, code))
    workspace = _workspace(workspace, ws_bytes, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    st = lib().ssm_ssd_bwd(Bsz, L, H, P, N, 1, code, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                           _ptr(z), _ptr(delta_bias), _ptr(h0), _ptr(dy), _ptr(dh_last), _ptr(out["dx"]),
                           _ptr(out["ddelta"]), _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["dD"]),
                           _ptr(out["dz"]), _ptr(out["ddelta_bias"]), _ptr(out["dh0"]), int(bool(delta_softplus)),
                           _ptr(workspace) if ws_bytes else None, ws_bytes, ctypes.c_void_p(s.cuda_stream))
    _check(st, "ssm_ssd_bwd")
    return out


def _rows(t, name, tokens, heads, d):
    """Elements from one token of t [B, L, heads, d] (tokens = (B, L)) or [B, heads, d] (tokens = (B,)) to the
    next, from its (shape, strides): t may be a part of a wider row (a slice of a joint projection's output) as
    long as its heads stand side by side and all tokens the same distance apart."""
    shape, st = t
    if tuple(shape) != (*tokens, heads, d):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {(*tokens, heads, d)}")
    if 0 in shape:
        return heads * d
    sizes = [(n, s) for n, s in zip(tokens, st) if n > 1]
    row = sizes[-1][1] if sizes else heads * d
    even = len(sizes) < 2 or sizes[0][1] == row * sizes[1][0]
    if (d > 1 and st[-1] != 1) or (heads > 1 and st[-2] != d) or not even or row < heads * d:
        raise ValueError(f"{name} must have its heads contiguous and its tokens evenly spaced (strides {tuple(st)})")
    return row


class _Sizes:
    """The ssm_linattn_shape of a call, its reference, and the sizes of its state, output and workspaces."""

    def __init__(self, shape):
        self.c = shape
        self.ref = ctypes.byref(shape)
        self.scale = shape.dk ** -0.5
        self.state = (shape.batch, shape.nheads, shape.dk, shape.dv)
        self.out = (shape.batch, shape.seqlen, shape.nheads, shape.dv)
        self.token = (shape.batch, shape.nheads, shape.dv)

    @functools.cached_property
    def fwd_bytes(self):
        return int(lib().ssm_linattn_workspace_bytes(self.ref))

    @functools.cached_property
    def bwd_bytes(self):
        return [int(lib().ssm_linattn_bwd_workspace_bytes(self.ref, i)) for i in (0, 1)]


@functools.lru_cache(maxsize=1024)
def _linattn_sizes(q, k, v, H, code):
    """From (shape, strides) of q, k and v, [B, L, heads, d] or [B, heads, d]."""
    n = len(q[0])
    if len(k[0]) != n or len(v[0]) != n or n not in (3, 4):
        raise ValueError(f"q, k and v must be [batch, {'seqlen, ' if n == 4 else ''}heads, dim]")
    head, dk, dv = tuple(q[0][:-2]), q[0][-1], v[0][-1]
    rows = [_rows(t, name, head, t[0][-2], d) for t, name, d in ((q, "q", dk), (k, "k", dk), (v, "v", dv))]
    return _Sizes(LinAttnShape(head[0], head[1] if n == 4 else 1, H, q[0][-2], k[0][-2], v[0][-2], dk, dv, *rows, code, 0))


def _linattn_call(q, k, v, log_decay, tokens, what):
    """Device, dtype and checked sizes of a call; tokens: 4 for [B, L, heads, d], 3 for [B, heads, d]."""
    import torch
    dev, dt = q.device, q.dtype
    if q.dim() != tokens:
        raise ValueError(f"q, k and v must be [batch, {'seqlen, ' if tokens == 4 else ''}heads, dim]")
    if log_decay.dim() != 1:
        raise ValueError("log_decay must be [nheads]")
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on the GPU only; tensors must be on a cuda device")
    code = _dtype_code(q)
    for t, name in ((k, "k"), (v, "v")):
        if t.dtype != dt:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dt}")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    _need(log_decay, "log_decay", log_decay.shape, torch.float32, dev)
    return dev, dt, _linattn_sizes((q.shape, q.stride()), (k.shape, k.stride()), (v.shape, v.stride()), log_decay.shape[0], code)


def _addr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    """torch's current HIP stream on the device, as a raw handle."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _elsewhere(device, stream):
    """None where a call runs as things are; else the context it has to run in: the tensors'
    device, and the stream given (what the call allocates then belongs to that stream)."""
    import torch
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    if stream is None and torch.cuda.current_device() == device.index:
        return None
    return torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)


def linattn_workspace_bytes(batch, seqlen, nheads, dk, dv, dtype="bf16") -> int:
    """Device workspace bytes of linattn_fwd for this shape (0: none)."""
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    s = LinAttnShape(batch, seqlen, nheads, nheads, nheads, nheads, dk, dv, 0, 0, 0, code, 0)
    return int(lib().ssm_linattn_workspace_bytes(ctypes.byref(s)))


def linattn_bwd_workspace_bytes(batch, seqlen, nheads, dk, dv, dtype="bf16", q_heads=None, k_heads=None,
                                v_heads=None, decay_grad=True) -> int:
    """Device workspace bytes of linattn_bwd for this shape; the head counts default to nheads."""
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    s = LinAttnShape(batch, seqlen, nheads, q_heads or nheads, k_heads or nheads, v_heads or nheads, dk, dv, 0, 0, 0, code, 0)
    return int(lib().ssm_linattn_bwd_workspace_bytes(ctypes.byref(s), int(bool(decay_grad))))


def linattn_fwd(q, k, v, log_decay, h0=None, *, scale=None, lengths=None, return_last_state=False, out=None,
                h_last=None, workspace=None, stream=None):
    """Linear attention with one decay per head, over a sequence:
    S_t = exp(log_decay) S_{t-1} + k_t v_t^T,  y_t = scale q_t^T S_t.

    q, k: [B, L, heads, dk];  v: [B, L, heads, dv] (all bf16, or all fp32; dk, dv <= 256);
    log_decay: [H] fp32, usually <= 0;  h0: [B, H, dk, dv] fp32.  The head counts of q, k and v
    each divide H: consecutive heads share a row.  q, k, v may be slices of one wider tensor
    (heads contiguous, tokens evenly spaced).  Every tensor but log_decay and lengths (which are
    copied where they do not) starts on 16 bytes; clone() a part that does not.  scale: default
    dk ** -0.5.  lengths: [B] int32, the tokens of each row, with padding behind them (y is zero
    there, the last state is the one after lengths[b] tokens).  Returns y [B, L, H, dv], or (y, h_last) when return_last_state.
    """
    import torch
    dev, dt, s = _linattn_call(q, k, v, log_decay, 4, "linattn_fwd")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return linattn_fwd(q, k, v, log_decay, h0, scale=scale, lengths=lengths, return_last_state=return_last_state,
                               out=out, h_last=h_last, workspace=workspace)
    _need(h0, "h0", s.state, torch.float32, dev)
    _need(lengths, "lengths", s.state[:1], torch.int32, dev)
    _need(out, "out", s.out, dt, dev)
    _need(h_last, "h_last", s.state, torch.float32, dev)
    if out is not None or h_last is not None:
        _written(out, h_last)
    if out is None:
        out = q.new_empty(s.out)   # (half the time of torch.empty)
    if return_last_state and h_last is None:
        h_last = log_decay.new_empty(s.state)
    log_decay, lengths = _aligned(log_decay), _aligned(lengths)
    need = s.fwd_bytes
    workspace = _workspace(workspace, need, dev)
    _check(lib().ssm_linattn_fwd(s.ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                                 s.scale if scale is None else scale, _addr(lengths), _addr(h0), _addr(h_last),
                                 out.data_ptr(), _addr(workspace) if need else None, need, _stream(dev)), "ssm_linattn_fwd")
    return (out, h_last) if return_last_state else out


def linattn_bwd(q, k, v, log_decay, h0=None, dy=None, dh_last=None, *, scale=None, lengths=None,
                need_dlog_decay=True, need_dh0=True, workspace=None, stream=None):
    """Gradients of a loss through linattn_fwd, given dy = dLoss/dy [B, L, H, dv] (q's dtype)
    and optionally dh_last = dLoss/dh_last [B, H, dk, dv] fp32.  Other arguments as linattn_fwd.

    Returns a dict: dq, dk, dv (contiguous, in the shapes and dtype of q, k, v; summed over the
    heads that share a row, zero in the padding), dlog_decay [H] fp32 (None when not needed: a
    fixed decay saves a third of the call) and dh0 [B, H, dk, dv] fp32 (None when not needed).
    """
    import torch
    dev, dt, s = _linattn_call(q, k, v, log_decay, 4, "linattn_bwd")
    if dy is None:
        raise ValueError("dy is required")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return linattn_bwd(q, k, v, log_decay, h0, dy, dh_last, scale=scale, lengths=lengths,
                               need_dlog_decay=need_dlog_decay, need_dh0=need_dh0, workspace=workspace)
    for t, n, shape, d in ((h0, "h0", s.state, torch.float32), (lengths, "lengths", s.state[:1], torch.int32),
                           (dy, "dy", s.out, dt), (dh_last, "dh_last", s.state, torch.float32)):
        _need(t, n, shape, d, dev)
    out = {"dq": q.new_empty(q.shape), "dk": k.new_empty(k.shape), "dv": v.new_empty(v.shape),
           "dlog_decay": log_decay.new_empty(log_decay.shape) if need_dlog_decay else None,
           "dh0": log_decay.new_empty(s.state) if need_dh0 else None}
    log_decay, lengths = _aligned(log_decay), _aligned(lengths)
    need = s.bwd_bytes[bool(need_dlog_decay)]
    workspace = _workspace(workspace, need, dev)
    _check(lib().ssm_linattn_bwd(s.ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                                 s.scale if scale is None else scale, _addr(lengths), _addr(h0), dy.data_ptr(),
                                 _addr(dh_last), out["dq"].data_ptr(), out["dk"].data_ptr(), out["dv"].data_ptr(),
                                 _addr(out["dlog_decay"]), _addr(out["dh0"]), _addr(workspace) if need else None, need,
                                 _stream(dev)), "ssm_linattn_bwd")
    return out


def linattn_update(h, q, k, v, log_decay, *, scale=None, out=None, stream=None):
    """One token of linattn_fwd: h [B, H, dk, dv] fp32 is updated in place; q, k [B, heads, dk],
    v [B, heads, dv], alignment as there; returns y [B, H, dv]."""
    import torch
    dev, dt, s = _linattn_call(q, k, v, log_decay, 3, "linattn_update")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return linattn_update(h, q, k, v, log_decay, scale=scale, out=out)
    _need(h, "h", s.state, torch.float32, dev)
    if out is None:
        out = q.new_empty(s.token)
    else:
        _need(out, "out", s.token, dt, dev)
        _written(out)
    torch.autograd.graph.increment_version(h)   # (as _written)
    decay = log_decay.data_ptr()
    if decay % 16:
        log_decay = log_decay.clone()
        decay = log_decay.data_ptr()
    _check(lib().ssm_linattn_update(s.ref, h.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), decay,
                                    s.scale if scale is None else scale, out.data_ptr(), _stream(dev)), "ssm_linattn_update")
    return out


@functools.lru_cache(maxsize=None)
def _linattn_function():
    import torch

    class _LinAttn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, log_decay, h0, scale, lengths, last):
            y, h = linattn_fwd(q, k, v, log_decay, h0, scale=scale, lengths=lengths, return_last_state=True) if last \
                else (linattn_fwd(q, k, v, log_decay, h0, scale=scale, lengths=lengths), None)
            ctx.save_for_backward(q, k, v, log_decay, h0, lengths)
            ctx.scale = scale
            return (y, h) if last else y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, gy, gh=None):
            q, k, v, log_decay, h0, lengths = ctx.saved_tensors
            need = ctx.needs_input_grad
            g = linattn_bwd(q, k, v, log_decay, h0, _gradient(gy), _gradient(gh),
                            scale=ctx.scale, lengths=lengths, need_dlog_decay=need[3], need_dh0=h0 is not None and need[4])
            return g["dq"], g["dk"], g["dv"], g["dlog_decay"], g["dh0"], None, None, None

    return _LinAttn


def linear_attention(q, k, v, log_decay, h0=None, *, scale=None, lengths=None, return_last_state=False):
    """Differentiable linear attention with one decay per head: linattn_fwd with a torch autograd
    backward through linattn_bwd (gradients for q, k, v, log_decay and h0).  Arguments as
    linattn_fwd; with return_last_state both outputs can be differentiated.

    In a captured graph, capture the forward and its backward together, and let no eager autograd
    graph of the same leaves live meanwhile: torch runs a leaf's accumulation on the stream that
    first used the leaf, which a capture cannot join."""
    return _linattn_function().apply(q, k, v, log_decay, h0, scale, lengths, bool(return_last_state))


def _norm_rows(x, groups, span, activation, what):
    """(batch, seqlen, dim) as the library takes them, the shape of the statistics, and silu: with span "token" every
    token is a batch row."""
    if x.dim() not in (2, 3):
        raise ValueError("x must be [batch, seqlen, dim] or [batch, dim]")
    if span not in ("token", "sequence"):
        raise ValueError(f"span {span!r} is neither 'token' nor 'sequence'")
    if activation not in ("none", "silu"):
        raise ValueError(f"activation {activation!r} is neither 'none' nor 'silu'")
    if x.device.type != "cuda":
        raise ValueError(f"{what} runs on the GPU only; tensors must be on a cuda device")
    head, dim = tuple(x.shape[:-1]), x.shape[-1]
    if span == "token":
        return (head[0] * (head[1] if len(head) == 2 else 1), 1, dim), (*head, groups), int(activation == "silu")
    return (head[0], head[1] if len(head) == 2 else 1, dim), (head[0], groups), int(activation == "silu")


def groupnorm_workspace_bytes(batch, seqlen, dim, groups, dtype="bf16", span="token", backward=False) -> int:
    """Device workspace bytes of groupnorm_fwd (or, with backward, groupnorm_bwd) for this shape (0: none)."""
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    n, length = (batch * seqlen, 1) if span == "token" else (batch, seqlen)
    return _groupnorm_bytes((n, length, dim), groups, code, int(bool(backward)))


@functools.lru_cache(maxsize=1024)
def _groupnorm_bytes(size, groups, code, backward):
    return int(lib().ssm_groupnorm_workspace_bytes(*size, groups, code, backward))


def groupnorm_fwd(x, groups, w=None, bias=None, z=None, *, span="token", activation="none", eps=1e-5,
                  return_stats=False, out=None, workspace=None, stream=None):
    """Group norm, channels last: u = (x - mean) / sqrt(var + eps) * w + bias, y = act(u) * silu(z).

    x, z: [B, L, D] or [B, D] (bf16 or fp32), the D channels in ``groups`` groups of consecutive
    ones; w, bias: [D] fp32.  span: the values that share a mean and variance, a group's channels
    of one token ("token": the norm after linear attention, a group per head) or of the whole
    sequence ("sequence").  activation: "none" or "silu".  Tensors are contiguous and start on 16
    bytes.  Returns y, or (y, mean, rstd) when
    return_stats: [B, L, groups] (or [B, groups]) fp32, what groupnorm_bwd reads.
    """
    import torch
    size, stats, silu = _norm_rows(x, groups, span, activation, "groupnorm_fwd")
    dev, dt, shape = x.device, x.dtype, x.shape
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return groupnorm_fwd(x, groups, w, bias, z, span=span, activation=activation, eps=eps, return_stats=return_stats,
                                 out=out, workspace=workspace)
    code = _dtype_code(x)
    _need(x, "x", shape, dt, dev)
    _need(z, "z", shape, dt, dev)
    _need(w, "w", shape[-1:], torch.float32, dev)
    _need(bias, "bias", shape[-1:], torch.float32, dev)
    _need(out, "out", shape, dt, dev)
    if out is None:
        out = x.new_empty(shape)
    else:
        _written(out)
    make = torch.empty if x.numel() else torch.zeros   # (the library leaves statistics of no values as they are)
    mean, rstd = (make(stats, dtype=torch.float32, device=dev) for _ in range(2)) if return_stats else (None, None)
    need = _groupnorm_bytes(size, groups, code, 0)
    workspace = _workspace(workspace, need, dev)
    _check(lib().ssm_groupnorm_fwd(*size, groups, code, x.data_ptr(), _addr(w), _addr(bias), _addr(z), eps, silu,
                                   out.data_ptr(), _addr(mean), _addr(rstd), _addr(workspace) if need else None, need,
                                   _stream(dev)), "ssm_groupnorm_fwd")
    return (out, mean, rstd) if return_stats else out


def groupnorm_bwd(x, groups, w=None, bias=None, z=None, dy=None, mean=None, rstd=None, *, span="token",
                  activation="none", need_dw=True, workspace=None, stream=None):
    """Gradients of a loss through groupnorm_fwd, given dy = dLoss/dy (x's shape and dtype) and
    the forward's mean and rstd.  Other arguments as groupnorm_fwd.

    Returns a dict: dx and dz (None without z) as x; dw (None without w) and dbias (None without a
    bias) [D] fp32, both None when need_dw is false.
    """
    import torch
    size, stats, silu = _norm_rows(x, groups, span, activation, "groupnorm_bwd")
    for t, n in ((dy, "dy"), (mean, "mean"), (rstd, "rstd")):
        if t is None:
            raise ValueError(f"{n} is required")
    dev, dt, shape = x.device, x.dtype, x.shape
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return groupnorm_bwd(x, groups, w, bias, z, dy, mean, rstd, span=span, activation=activation, need_dw=need_dw,
                                 workspace=workspace)
    code = _dtype_code(x)
    for t, n, s, d in ((x, "x", shape, dt), (z, "z", shape, dt), (dy, "dy", shape, dt), (w, "w", shape[-1:], torch.float32),
                       (bias, "bias", shape[-1:], torch.float32), (mean, "mean", stats, torch.float32),
                       (rstd, "rstd", stats, torch.float32)):
        _need(t, n, s, d, dev)
    out = {"dx": x.new_empty(shape), "dz": x.new_empty(shape) if z is not None else None,
           "dw": w.new_empty(shape[-1:]) if w is not None and need_dw else None,
           "dbias": bias.new_empty(shape[-1:]) if bias is not None and need_dw else None}
    need = _groupnorm_bytes(size, groups, code, 1)
    workspace = _workspace(workspace, need, dev)
    _check(lib().ssm_groupnorm_bwd(*size, groups, code, x.data_ptr(), _addr(w), _addr(bias), _addr(z), silu, dy.data_ptr(),
                                   mean.data_ptr(), rstd.data_ptr(), out["dx"].data_ptr(), _addr(out["dw"]),
                                   _addr(out["dbias"]), _addr(out["dz"]), _addr(workspace) if need else None, need,
                                   _stream(dev)), "ssm_groupnorm_bwd")
    return out


@functools.lru_cache(maxsize=None)
def _groupnorm_function():
    import torch

    class _GroupNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, groups, w, bias, z, span, activation, eps):
            y, mean, rstd = groupnorm_fwd(x, groups, w, bias, z, span=span, activation=activation, eps=eps, return_stats=True)
            ctx.save_for_backward(x, w, bias, z, mean, rstd)
            ctx.how = groups, span, activation
            return y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, gy):
            x, w, bias, z, mean, rstd = ctx.saved_tensors
            groups, span, activation = ctx.how
            g = groupnorm_bwd(x, groups, w, bias, z, _gradient(gy), mean, rstd, span=span, activation=activation,
                              need_dw=ctx.needs_input_grad[2] or ctx.needs_input_grad[3])
            return g["dx"], None, g["dw"], g["dbias"], g["dz"], None, None, None

    return _GroupNorm


def group_norm(x, groups, w=None, bias=None, z=None, *, span="token", activation="none", eps=1e-5):
    """Differentiable group norm, channels last: groupnorm_fwd with a torch autograd backward
    through groupnorm_bwd (gradients for x, w, bias and z).  Arguments as groupnorm_fwd; captured
    graphs as linear_attention."""
    return _groupnorm_function().apply(x, groups, w, bias, z, span, activation, eps)


def rotary_freqs(rot, base=10000.0, *, scaling="none", factor=1.0, context=4096, fast=32.0, slow=1.0, device="cuda"):
    """(freqs, magnitude) of rotary_fwd and qknorm_fwd for ``rot`` turning columns: freqs[j] = base ** (-2 j / rot) radians
    a position, [rot / 2] fp64 on ``device``; to reach contexts ``factor`` times as long as the ``context`` positions of training,
    scaled: "linear" (every frequency divided by the factor), "base" (a larger base, so that the slowest pair is
    divided by the factor and the fastest stays), or "bands" (pairs that turn ``fast`` times or more over the context stay,
    those that turn ``slow`` times or less are divided, in between a linear mix of both; the magnitude is then
    0.1 log(factor) + 1, else 1)."""
    import math
    import torch
    if rot < 2 or rot % 2:
        raise ValueError(f"rot={rot} must be even and >= 2")
    if not (base > 0 and factor >= 1 and context > 0 and fast > slow > 0):
        raise ValueError("base and context must be positive, factor >= 1 and fast > slow > 0")
    if scaling not in ("none", "linear", "base", "bands"):
        raise ValueError(f"scaling {scaling!r} is not one of 'none', 'linear', 'base', 'bands'")
    j = torch.arange(rot // 2, dtype=torch.float64) / (rot // 2)
    if scaling == "base" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f, magnitude = torch.pow(torch.tensor(float(base), dtype=torch.float64), -j), 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        stay = ((context * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f, magnitude = f * stay + f / factor * (1.0 - stay), 0.1 * math.log(factor) + 1.0
    return f.to(device), magnitude


class _RotarySizes:
    """The ssm_rotary_shape of a call, its reference, and the shapes of its outputs and workspace."""

    def __init__(self, shape, q, k):
        self.c = shape
        self.ref = ctypes.byref(shape)
        self.q, self.k = q, k
        self.w = (shape.dim,)

    @functools.cached_property
    def bwd_bytes(self):
        return int(lib().ssm_qknorm_bwd_workspace_bytes(self.ref))


@functools.lru_cache(maxsize=1024)
def _rotary_sizes(q, k, positions, pairs, layout, code):
    """From (shape, strides) of q and k ([B, L, heads, dim] or [B, heads, dim]; k may be None) and the shape of positions."""
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout {layout!r} is neither 'half' nor 'interleaved'")
    n = len(q[0])
    if n not in (3, 4) or (k is not None and len(k[0]) != n):
        raise ValueError("q and k must be [batch, seqlen, heads, dim] or [batch, heads, dim]")
    head, d = tuple(q[0][:-2]), q[0][-1]
    qr = _rows(q, "q", head, q[0][-2], d)
    kr = _rows(k, "k", head, k[0][-2], d) if k is not None else 0
    if pairs and positions not in (head, head[-1:]):
        raise ValueError(f"positions has shape {positions}, expected {head}" + (f" or {head[-1:]}" if n == 4 else ""))
    if 2 * pairs > d:
        raise ValueError(f"{pairs} frequencies turn {2 * pairs} columns, but heads have {d}")
    tokens = head[0] * (head[1] if n == 4 else 1)
    period = positions[0] if pairs and positions != head else 0
    return _RotarySizes(RotaryShape(tokens, period, q[0][-2], k[0][-2] if k is not None else 0, d, 2 * pairs, qr, kr,
                                    int(layout == "interleaved"), code), tuple(q[0]), tuple(k[0]) if k is not None else None)


def _rotary_call(q, k, positions, freqs, layout, what):
    import torch
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on the GPU only; tensors must be on a cuda device")
    code = _dtype_code(q)
    if k is not None and (k.dtype != dt or k.device != dev):
        raise (TypeError if k.dtype != dt else ValueError)(f"k is {k.dtype} on {k.device}, q {dt} on {dev}")
    if (positions is None) != (freqs is None):
        raise ValueError("positions and freqs go together")
    shape, pairs = (), 0
    if freqs is not None:
        _need(freqs, "freqs", freqs.shape[:1] if freqs.dim() else (1,), torch.float64, dev)
        shape, pairs = tuple(positions.shape), freqs.shape[0]
        _need(positions, "positions", shape, torch.int32, dev)
    return dev, dt, _rotary_sizes((q.shape, q.stride()), None if k is None else (k.shape, k.stride()), shape, pairs, layout, code)


def _rotary_outs(out, q, k, s, dt, dev):
    if out is None:
        return q.new_empty(s.q), None if k is None else k.new_empty(s.k)
    if not isinstance(out, (tuple, list)) or len(out) != 2 or out[0] is None or (out[1] is None) != (k is None):
        raise ValueError("out must be a pair, of q's output and of k's (None without k)")
    _need(out[0], "out[0]", s.q, dt, dev)
    _need(out[1], "out[1]", s.k, dt, dev)
    _written(*out)
    return tuple(out)


def rotary_fwd(q, k=None, positions=None, freqs=None, *, layout="half", magnitude=1.0, out=None, stream=None, _back=0):
    """Rotary positions: pair j of each head's first 2 len(freqs) columns turned by positions * freqs[j], times
    magnitude; the columns behind them as they are.

    q, k: [B, L, heads, dim], or [B, heads, dim] for single tokens (bf16, or fp32; dim <= 256; k may
    be None), which may be slices of a joint projection's output (heads side by side, tokens evenly
    spaced; rows and addresses in multiples of 16 bytes are the fast ones).  positions: int32, one for
    every token, or [L] for all rows alike; freqs: [pairs] fp64 (rotary_freqs).  layout: pairs are columns
    (j, j + len(freqs)) ("half") or (2 j, 2 j + 1) ("interleaved").  Returns (q, k) turned, contiguous, or
    q alone where k is None.
    """
    if freqs is None:
        raise ValueError("positions and freqs are required")
    dev, dt, s = _rotary_call(q, k, positions, freqs, layout, "rotary_fwd")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return rotary_fwd(q, k, positions, freqs, layout=layout, magnitude=magnitude, out=out, _back=_back)
    qo, ko = _rotary_outs(out, q, k, s, dt, dev)
    _check(lib().ssm_rotary_fwd(s.ref, q.data_ptr(), _addr(k), positions.data_ptr(), freqs.data_ptr(), magnitude, _back,
                                qo.data_ptr(), _addr(ko), _stream(dev)), "ssm_rotary_fwd")
    return qo if k is None else (qo, ko)


def rotary_bwd(dq, dk=None, positions=None, freqs=None, *, layout="half", magnitude=1.0, out=None, stream=None):
    """Gradients for rotary_fwd's q and k from those of its outputs: the same turn by the opposite angles."""
    return rotary_fwd(dq, dk, positions, freqs, layout=layout, magnitude=magnitude, out=out, stream=stream, _back=1)


def qknorm_fwd(q, k=None, wq=None, wk=None, positions=None, freqs=None, *, eps=1e-6, layout="half", magnitude=1.0, out=None,
               stream=None):
    """An RMS norm of every head, u = x / sqrt(mean(x^2) + eps) * w, and rotary_fwd of the normed rows in
    the same pass.  wq, wk: [dim] fp32, for the heads of q and of k (None: ones); positions and freqs None: the
    norm alone.  Other arguments, and what is returned, as rotary_fwd."""
    import torch
    dev, dt, s = _rotary_call(q, k, positions, freqs, layout, "qknorm_fwd")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return qknorm_fwd(q, k, wq, wk, positions, freqs, eps=eps, layout=layout, magnitude=magnitude, out=out)
    _need(wq, "wq", s.w, torch.float32, dev)
    _need(wk, "wk", s.w, torch.float32, dev)
    qo, ko = _rotary_outs(out, q, k, s, dt, dev)
    _check(lib().ssm_qknorm_fwd(s.ref, q.data_ptr(), _addr(k), _addr(wq), _addr(wk), _addr(positions), _addr(freqs), eps,
                                magnitude, qo.data_ptr(), _addr(ko), _stream(dev)), "ssm_qknorm_fwd")
    return qo if k is None else (qo, ko)


def qknorm_bwd_workspace_bytes(tokens, dim) -> int:
    """Device workspace bytes of qknorm_bwd (with gradients of weights) for this many tokens of heads of dim columns."""
    s = RotaryShape(tokens, 0, 1, 0, dim, 0, 0, 0, 0, 0)
    return int(lib().ssm_qknorm_bwd_workspace_bytes(ctypes.byref(s)))


def qknorm_bwd(q, k=None, wq=None, wk=None, positions=None, freqs=None, dq_out=None, dk_out=None, *, eps=1e-6, layout="half",
               magnitude=1.0, need_dw=True, workspace=None, stream=None):
    """Gradients of a loss through qknorm_fwd, given its inputs and dq_out, dk_out = the gradients of its outputs
    (contiguous, their shapes and dtype).

    Returns a dict: dq, dk (None without k) as q and k, contiguous; dwq, dwk [dim] fp32 (None without that weight, or when
    need_dw is false).
    """
    import torch
    dev, dt, s = _rotary_call(q, k, positions, freqs, layout, "qknorm_bwd")
    if dq_out is None or (dk_out is None) != (k is None):
        raise ValueError("dq_out is required, and dk_out where there is a k")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return qknorm_bwd(q, k, wq, wk, positions, freqs, dq_out, dk_out, eps=eps, layout=layout, magnitude=magnitude,
                              need_dw=need_dw, workspace=workspace)
    _need(wq, "wq", s.w, torch.float32, dev)
    _need(wk, "wk", s.w, torch.float32, dev)
    _need(dq_out, "dq_out", s.q, dt, dev)
    _need(dk_out, "dk_out", s.k, dt, dev)
    out = {"dq": q.new_empty(s.q), "dk": None if k is None else k.new_empty(s.k),
           "dwq": None if wq is None or not need_dw else wq.new_empty(s.w),
           "dwk": None if wk is None or not need_dw else wk.new_empty(s.w)}
    need = 0 if out["dwq"] is None and out["dwk"] is None else s.bwd_bytes
    workspace = _workspace(workspace, need, dev)
    _check(lib().ssm_qknorm_bwd(s.ref, q.data_ptr(), _addr(k), _addr(wq), _addr(wk), _addr(positions), _addr(freqs), eps,
                                magnitude, dq_out.data_ptr(), _addr(dk_out), out["dq"].data_ptr(), _addr(out["dk"]),
                                _addr(out["dwq"]), _addr(out["dwk"]), _addr(workspace) if need else None, need, _stream(dev)),
           "ssm_qknorm_bwd")
    return out


@functools.lru_cache(maxsize=None)
def _rotary_functions():
    import torch

    def whole(g, shape, like):
        """The gradient of an output that nothing was made of is zero."""
        return _gradient(g) if g is not None else like.new_zeros(shape)

    class _Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, positions, freqs, layout, magnitude):
            ctx.save_for_backward(positions, freqs)
            ctx.set_materialize_grads(False)
            ctx.how = {"layout": layout, "magnitude": magnitude}
            return rotary_fwd(q, k, positions, freqs, **ctx.how)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, gq, gk=None):
            positions, freqs = ctx.saved_tensors
            turned = [None, None]
            if gq is not None and gk is not None and ctx.needs_input_grad[0] and ctx.needs_input_grad[1]:
                turned = rotary_bwd(_gradient(gq), _gradient(gk), positions, freqs, **ctx.how)
            else:
                for i, g in enumerate((gq, gk)):
                    if g is not None and ctx.needs_input_grad[i]:
                        turned[i] = rotary_bwd(_gradient(g), None, positions, freqs, **ctx.how)
            return turned[0], turned[1], None, None, None, None

    class _QKNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, wq, wk, positions, freqs, eps, layout, magnitude):
            ctx.save_for_backward(q, k, wq, wk, positions, freqs)
            ctx.set_materialize_grads(False)
            ctx.how = {"eps": eps, "layout": layout, "magnitude": magnitude}
            return qknorm_fwd(q, k, wq, wk, positions, freqs, **ctx.how)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, gq, gk=None):
            q, k, wq, wk, positions, freqs = ctx.saved_tensors
            g = qknorm_bwd(q, k, wq, wk, positions, freqs, whole(gq, q.shape, q), None if k is None else whole(gk, k.shape, k),
                           need_dw=ctx.needs_input_grad[2] or ctx.needs_input_grad[3], **ctx.how)
            return g["dq"], g["dk"], g["dwq"], g["dwk"], None, None, None, None, None

    return _Rotary, _QKNorm


def rotary(q, k, positions, freqs, *, layout="half", magnitude=1.0):
    """Differentiable rotary positions: rotary_fwd with a torch autograd backward through rotary_bwd (gradients for q
    and k).  Arguments as rotary_fwd; captured graphs as linear_attention."""
    return _rotary_functions()[0].apply(q, k, positions, freqs, layout, magnitude)


def qk_norm(q, k, wq=None, wk=None, positions=None, freqs=None, *, eps=1e-6, layout="half", magnitude=1.0):
    """Differentiable norms of every head of q and k with their rotary positions: qknorm_fwd with a torch autograd
    backward through qknorm_bwd (gradients for q, k, wq and wk).  Arguments as qknorm_fwd; captured graphs as
    linear_attention."""
    return _rotary_functions()[1].apply(q, k, wq, wk, positions, freqs, eps, layout, magnitude)


class _SsdConvSizes:
    """The ssm_ssdconv_shape of a call, its reference, and the shapes of its tensors and workspace."""

    def __init__(self, c, token):
        self.c = c
        self.ref = ctypes.byref(c)
        self.channels = c.nheads * c.headdim + 2 * c.ngroups * c.dstate
        self.heads, self.token = (c.nheads,), token
        self.w, self.bias = (self.channels, c.width), (self.channels,)
        self.y = (c.tokens, c.nheads, c.headdim)
        self.conv_state = (c.nslots, self.channels, c.width - 1)
        self.seqs, self.offsets = (c.sequences,), (c.sequences + 1,)

    @functools.cached_property
    def bytes(self):
        L = lib()
        return int((L.ssm_ssdconv_update_workspace_bytes if self.token else L.ssm_ssdconv_workspace_bytes)(self.ref))


def _row(t, name, width):
    """Elements from one row of t [rows, width] (or [rows, heads, dim], one row of width values) to the next."""
    shape, st = t
    if 0 in shape:
        return width
    inner = [(n, s) for n, s in zip(shape[1:], st[1:]) if n > 1]
    at = 1
    for n, s in reversed(inner):
        if s != at:
            raise ValueError(f"{name} must have rows of contiguous values (strides {tuple(st)})")
        at *= n
    row = st[0] if shape[0] > 1 else width
    if row < width:
        raise ValueError(f"{name}'s rows overlap (strides {tuple(st)})")
    return row


@functools.lru_cache(maxsize=4096)
def _ssdconv_sizes(xbc, delta, z, h, w, sequences, max_seqlen, token, code):
    """From (shape, strides) of xbc, delta and z, and the shapes of h and w."""
    if len(xbc[0]) != 2 or len(h) != 4 or len(w) != 2:
        raise ValueError("xbc must be [tokens, channels], h [slots, nheads, headdim, dstate] and w [channels, width]")
    T, C = xbc[0]
    nslots, H, P, N = h
    G, rest = divmod(C - H * P, 2 * N) if N else (0, 1)
    if rest or G < 1:
        raise ValueError(f"xbc has {C} channels: not nheads * headdim + 2 * ngroups * dstate = {H} * {P} + 2 * ngroups * {N}")
    if tuple(delta[0]) != (T, H):
        raise ValueError(f"delta has shape {tuple(delta[0])}, expected {(T, H)}")
    if z is not None and tuple(z[0]) != (T, H, P):
        raise ValueError(f"z has shape {tuple(z[0])}, expected {(T, H, P)}")
    c = SsdConvShape(T, T if token else sequences, max_seqlen, H, P, N, G, w[1], nslots, _row(xbc, "xbc", C),
                     0 if z is None else _row(z, "z", H * P), _row(delta, "delta", H), code, 0)
    return _SsdConvSizes(c, token)


def ssdconv_workspace_bytes(tokens, sequences, nheads, headdim, dstate, ngroups=1, width=4, dtype="bf16", max_seqlen=0,
                            update=False) -> int:
    """Device workspace bytes of ssdconv_fwd (or, with update, ssdconv_update) for this shape (0: none)."""
    code = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    c = SsdConvShape(tokens, sequences, max_seqlen, nheads, headdim, dstate, ngroups, width, sequences, 0, 0, 0, code, 0)
    L = lib()
    return int((L.ssm_ssdconv_update_workspace_bytes if update else L.ssm_ssdconv_workspace_bytes)(ctypes.byref(c)))


def _ssdconv_call(xbc, delta, A, w, h, conv_state, slots, sequences, bias, D, z, delta_bias, max_seqlen, out, what):
    import torch
    dev, dt = xbc.device, xbc.dtype
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on the GPU only; tensors must be on a cuda device")
    code = _dtype_code(xbc)
    for t, name in ((delta, "delta"), (z, "z")):
        if t is not None and t.dtype != dt:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dt}")
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    s = _ssdconv_sizes((xbc.shape, xbc.stride()), (delta.shape, delta.stride()), None if z is None else (z.shape, z.stride()),
                       h.shape, w.shape, sequences, max_seqlen, what == "ssdconv_update", code)
    f32 = torch.float32
    _need(A, "A", s.heads, f32, dev)
    _need(w, "w", s.w, f32, dev)
    _need(bias, "bias", s.bias, f32, dev)
    _need(D, "D", s.heads, f32, dev)
    _need(delta_bias, "delta_bias", s.heads, f32, dev)
    _need(h, "h", h.shape, f32, dev)
    if conv_state is None and s.c.width > 1:
        raise ValueError("conv_state is required for a filter of more than one column")
    _need(conv_state, "conv_state", s.conv_state, dt, dev)
    _need(slots, "slots", s.seqs, torch.int32, dev)
    _need(out, "out", s.y, dt, dev)
    return dev, s


def ssdconv_fwd(xbc, delta, A, w, h, conv_state, offsets, slots=None, *, bias=None, D=None, z=None, delta_bias=None,
                delta_softplus=False, fresh=None, max_seqlen=None, out=None, workspace=None, stream=None):
    """A Mamba-2 layer's mixer over packed sequences whose states lie in a pool: the causal convolution (+ SiLU) of
    conv1d_fwd over the channels of x, B and C, and the multi-head scan of ssd_fwd behind it.  (For serving: no gradients;
    those two have them.)

    xbc: [T, H P + 2 G N], a row (x [H, P], B [G, N], C [G, N]) for every token;  delta: [T, H];  z: [T, H, P] (all
    bf16, or all fp32), each possibly a slice of a joint projection's output (contiguous rows, evenly spaced);
    A, D, delta_bias: [H] fp32;  w: [channels, W] fp32 (W <= 4), bias: [channels] fp32.  h: [slots, H, P, N]
    fp32 (N <= 128) and conv_state: [slots, channels, W - 1] (xbc's dtype) are read and updated in place.  offsets: [S + 1]
    int32: sequence s has the rows offsets[s] .. offsets[s + 1] - 1 (other rows of y are not written).
    slots: [S] int32, no two alike (default: sequence s has slot s); outside the pool (-1): from zeros, and not
    kept.  fresh: [S] bool, where a sequence starts from zeros whatever its slot holds.  max_seqlen: the longest sequence's
    tokens, as the host knows them (they decide how sequences are split); default T.  Returns y [T, H, P].
    """
    import torch
    if offsets.dim() != 1 or not offsets.shape[0]:
        raise ValueError("offsets must be [sequences + 1]")
    S = offsets.shape[0] - 1
    dev, s = _ssdconv_call(xbc, delta, A, w, h, conv_state, slots, S, bias, D, z, delta_bias, int(max_seqlen or 0), out, "ssdconv_fwd")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return ssdconv_fwd(xbc, delta, A, w, h, conv_state, offsets, slots, bias=bias, D=D, z=z, delta_bias=delta_bias,
                               delta_softplus=delta_softplus, fresh=fresh, max_seqlen=max_seqlen, out=out, workspace=workspace)
    _need(offsets, "offsets", s.offsets, torch.int32, dev)
    _need(fresh, "fresh", s.seqs, torch.bool, dev)
    if out is None:
        out = xbc.new_empty(s.y)
    else:
        _written(out)
    _written(h, conv_state)
    need = s.bytes
    workspace = _workspace(workspace, need, dev)
    _check(lib().ssm_ssdconv_fwd(s.ref, xbc.data_ptr(), delta.data_ptr(), A.data_ptr(), w.data_ptr(), _addr(bias), _addr(D), _addr(z),
                                 _addr(delta_bias), int(bool(delta_softplus)), offsets.data_ptr(), _addr(slots), _addr(fresh),
                                 h.data_ptr(), _addr(conv_state), out.data_ptr(), _addr(workspace) if need else None, need,
                                 _stream(dev)), "ssm_ssdconv_fwd")
    return out


def ssdconv_update(xbc, delta, A, w, h, conv_state, slots=None, *, bias=None, D=None, z=None, delta_bias=None,
                   delta_softplus=False, out=None, workspace=None, stream=None):
    """One token of every sequence of ssdconv_fwd: xbc [S, channels], delta [S, H], z [S, H, P]; h and conv_state are
    updated in place.  Other arguments as there.  Returns y [S, H, P]."""
    dev, s = _ssdconv_call(xbc, delta, A, w, h, conv_state, slots, 0, bias, D, z, delta_bias, 0, out, "ssdconv_update")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return ssdconv_update(xbc, delta, A, w, h, conv_state, slots, bias=bias, D=D, z=z, delta_bias=delta_bias,
                                  delta_softplus=delta_softplus, out=out, workspace=workspace)
    if out is None:
        out = xbc.new_empty(s.y)
    else:
        _written(out)
    _written(h, conv_state)
    need = s.bytes
    workspace = _workspace(workspace, need, dev)
    _check(lib().ssm_ssdconv_update(s.ref, xbc.data_ptr(), delta.data_ptr(), A.data_ptr(), w.data_ptr(), _addr(bias), _addr(D),
                                    _addr(z), _addr(delta_bias), int(bool(delta_softplus)), _addr(slots), h.data_ptr(),
                                    _addr(conv_state), out.data_ptr(), _addr(workspace) if need else None, need, _stream(dev)),
           "ssm_ssdconv_update")
    return out
