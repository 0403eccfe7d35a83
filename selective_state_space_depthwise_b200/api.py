"""PyTorch-facing calls of the C ABI (include/ssm.h).

Each function reads sizes and strides off the tensors, allocates missing
outputs with torch (device memory is PyTorch's job here), and makes exactly
one C call on the current CUDA stream. Every step of the block core runs in
the library's CUDA kernels; tensors that are not on a CUDA device are
rejected -- there is no CPU path.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

_DTYPES = {torch.float32: _lib.SSM_F32, torch.bfloat16: _lib.SSM_BF16}
_DISC = {"euler": _lib.SSM_DISC_EULER_B, "euler_b": _lib.SSM_DISC_EULER_B, "zoh": _lib.SSM_DISC_ZOH}
PARAM_NAMES = ("conv_w", "conv_b", "w_dt", "dt_bias", "A_log", "D")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need_cuda(name, t, device):
    if t is None:
        return
    if not t.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA tensor: the block core has no CPU path")
    if t.device != device:
        raise RuntimeError(f"{name} is on {t.device}, expected {device}")


def _weights(params, E, device):
    for n in PARAM_NAMES:
        t = params[n]
        _need_cuda(n, t, device)
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous float32")
    if params["conv_w"].shape != (E, 4) or params["A_log"].shape != (E, 16):
        raise ValueError("conv_w must be [E, 4] and A_log [E, 16]")
    for n in ("conv_b", "w_dt", "dt_bias", "D"):
        if params[n].shape != (E,):
            raise ValueError(f"{n} must be [E]")
    w = _lib.SsmWeights()
    for n in PARAM_NAMES:
        setattr(w, n, params[n].data_ptr())
    return w


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _tuning_ref(tuning):
    """ssm_tuning from a dict {"kernel": k, "decay_path": d} (None: defaults)."""
    if not tuning:
        return None
    unknown = set(tuning) - {"kernel", "decay_path"}
    if unknown:
        raise ValueError(f"unknown tuning keys {sorted(unknown)} (kernel, decay_path)")
    return ctypes.byref(_lib.SsmTuning(int(tuning.get("kernel", 0)), int(tuning.get("decay_path", 0))))


def make_dims(batch, seqlen, E, io_dtype, dt_min=1e-4, dt_max=1.0, discretization="euler", **strides):
    d = _lib.SsmDims()
    d.batch, d.seqlen, d.d_inner, d.d_state, d.d_conv = batch, seqlen, E, 16, 4
    d.dt_min, d.dt_max = dt_min, dt_max
    d.io_dtype = _DTYPES[io_dtype] if isinstance(io_dtype, torch.dtype) else int(io_dtype)
    d.discretization = _DISC[discretization]
    for k, v in strides.items():
        setattr(d, k, int(v))
    return d


def workspace_bytes(batch, seqlen, E, io_dtype=torch.bfloat16) -> int:
    lib = _lib.load()
    return int(lib.ssm_prefill_workspace_bytes(ctypes.byref(make_dims(batch, seqlen, E, io_dtype))))


def prefill_kernel(batch, seqlen, E, io_dtype=torch.bfloat16, discretization="euler", tuning=None,
                   num_sms=0) -> int:
    """The prefill kernel (3, 4 or 5) `prefill` launches for this shape and
    tuning on a GPU of num_sms SMs (0: the current device's); 0 where the call
    would be rejected. Host-only for num_sms > 0."""
    lib = _lib.load()
    dims = make_dims(batch, seqlen, E, io_dtype, discretization=discretization)
    return int(lib.ssm_prefill_kernel(ctypes.byref(dims), _tuning_ref(tuning), int(num_sms)))


def prefill(x, z, B, C, dt_raw, params, *, conv_cache_in=None, ssm_state_in=None, y=None, conv_cache_out=None,
            ssm_state_out=None, dt_min=1e-4, dt_max=1.0, discretization="euler", tuning=None, stream=None):
    """Full-sequence block core. x, z: [b, L, E] (last dim contiguous; token and
    sequence strides are passed through); B, C: [b, L, 16]; dt_raw: [b, L].
    Returns (y [b, L, E], conv_cache_out [b, 3, E], ssm_state_out [b, E, 16])."""
    lib = _lib.load()
    b, L, E = x.shape
    dev = x.device
    for n, t in (("x", x), ("z", z), ("B", B), ("C", C), ("dt_raw", dt_raw), ("conv_cache_in", conv_cache_in),
                 ("ssm_state_in", ssm_state_in), ("y", y), ("conv_cache_out", conv_cache_out),
                 ("ssm_state_out", ssm_state_out)):
        _need_cuda(n, t, dev)
    if x.dtype not in _DTYPES or z.dtype != x.dtype:
        raise ValueError("x and z must share an io dtype (float32 or bfloat16)")
    if z.shape != (b, L, E) or B.shape != (b, L, 16) or C.shape != (b, L, 16) or dt_raw.shape != (b, L):
        raise ValueError("shape mismatch: z [b,L,E], B/C [b,L,16], dt_raw [b,L]")
    if x.stride(2) != 1 or z.stride(2) != 1 or B.stride(2) != 1 or dt_raw.stride(1) != 1:
        raise ValueError("the innermost dimension of x, z, B, C, dt_raw must be contiguous")
    if B.stride() != C.stride():
        raise ValueError("B and C must share strides")
    if y is None:
        y = torch.empty((b, L, E), dtype=x.dtype, device=dev)
    if conv_cache_out is None:
        conv_cache_out = torch.empty((b, 3, E), dtype=x.dtype, device=dev)
    if ssm_state_out is None:
        ssm_state_out = torch.empty((b, E, 16), dtype=torch.float32, device=dev)
    for n, t, shp, dt in (("conv_cache_out", conv_cache_out, (b, 3, E), x.dtype),
                          ("ssm_state_out", ssm_state_out, (b, E, 16), torch.float32),
                          ("conv_cache_in", conv_cache_in, (b, 3, E), x.dtype),
                          ("ssm_state_in", ssm_state_in, (b, E, 16), torch.float32)):
        if t is not None and (t.shape != shp or t.dtype != dt or not t.is_contiguous()):
            raise ValueError(f"{n} must be a contiguous {dt} tensor of shape {shp}")
    if y.shape != (b, L, E) or y.dtype != x.dtype or y.stride(2) != 1:
        raise ValueError("y must be [b, L, E] in the io dtype with a contiguous last dim")
    dims = make_dims(b, L, E, x.dtype, dt_min, dt_max, discretization,
                     x_tok_stride=x.stride(1), x_seq_stride=x.stride(0), z_tok_stride=z.stride(1),
                     z_seq_stride=z.stride(0), y_tok_stride=y.stride(1), y_seq_stride=y.stride(0),
                     bc_tok_stride=B.stride(1), bc_seq_stride=B.stride(0), dt_seq_stride=dt_raw.stride(0))
    w = _weights(params, E, dev)
    ws = int(lib.ssm_prefill_workspace_bytes(ctypes.byref(dims)))
    work = torch.empty(ws, dtype=torch.uint8, device=dev) if ws else None
    st = lib.ssm_prefill_ex(ctypes.byref(dims), ctypes.byref(w), _ptr(x), _ptr(z), _ptr(B), _ptr(C), _ptr(dt_raw),
                            _ptr(conv_cache_in), _ptr(ssm_state_in), _ptr(y), _ptr(conv_cache_out),
                            _ptr(ssm_state_out), _ptr(work), ws, _tuning_ref(tuning), _stream(stream))
    _lib.check(st)
    return y, conv_cache_out, ssm_state_out


def host_workspace_bytes(batch, seqlen, E, io_dtype=torch.bfloat16, chunk_tokens=0) -> int:
    lib = _lib.load()
    return int(lib.ssm_prefill_host_workspace_bytes(ctypes.byref(make_dims(batch, seqlen, E, io_dtype)),
                                                    int(chunk_tokens)))


def prefill_host(x, z, B, C, dt_raw, params, *, conv_cache_in=None, ssm_state_in=None, y=None, conv_cache_out=None,
                 ssm_state_out=None, dt_min=1e-4, dt_max=1.0, discretization="euler", chunk_tokens=0, workspace=None,
                 stream=None, static_scratch=False):
    """Full-sequence block core with the token tensors in host memory
    (ssm_prefill_host): x, z, B, C, dt_raw and y are pinned CPU tensors
    (pageable ones are refused), shaped and strided as for `prefill`; the parameters and
    the caches are CUDA tensors on the current device. The copies and kernels
    are only enqueued: synchronise `stream` before reading y. With
    static_scratch=True the call goes to ssm_prefill_host_static, which takes
    no workspace and allocates nothing (its chunk buffers are the library's
    static device scratch).
    Returns (y [b, L, E] on the host, conv_cache_out, ssm_state_out)."""
    lib = _lib.load()
    b, L, E = x.shape
    dev = params["A_log"].device
    for n, t in (("x", x), ("z", z), ("B", B), ("C", C), ("dt_raw", dt_raw), ("y", y)):
        if t is not None and t.is_cuda:
            raise RuntimeError(f"{n} must be a host tensor for prefill_host (use prefill for device tensors)")
    for n, t in (("conv_cache_in", conv_cache_in), ("ssm_state_in", ssm_state_in),
                 ("conv_cache_out", conv_cache_out), ("ssm_state_out", ssm_state_out)):
        _need_cuda(n, t, dev)
    if x.dtype not in _DTYPES or z.dtype != x.dtype:
        raise ValueError("x and z must share an io dtype (float32 or bfloat16)")
    if z.shape != (b, L, E) or B.shape != (b, L, 16) or C.shape != (b, L, 16) or dt_raw.shape != (b, L):
        raise ValueError("shape mismatch: z [b,L,E], B/C [b,L,16], dt_raw [b,L]")
    if x.stride(2) != 1 or z.stride(2) != 1 or B.stride(2) != 1 or dt_raw.stride(1) != 1:
        raise ValueError("the innermost dimension of x, z, B, C, dt_raw must be contiguous")
    if B.stride() != C.stride():
        raise ValueError("B and C must share strides")
    if y is None:
        y = torch.empty((b, L, E), dtype=x.dtype, pin_memory=True)
    if conv_cache_out is None:
        conv_cache_out = torch.empty((b, 3, E), dtype=x.dtype, device=dev)
    if ssm_state_out is None:
        ssm_state_out = torch.empty((b, E, 16), dtype=torch.float32, device=dev)
    if y.shape != (b, L, E) or y.dtype != x.dtype or y.stride(2) != 1:
        raise ValueError("y must be [b, L, E] in the io dtype with a contiguous last dim")
    dims = make_dims(b, L, E, x.dtype, dt_min, dt_max, discretization,
                     x_tok_stride=x.stride(1), x_seq_stride=x.stride(0), z_tok_stride=z.stride(1),
                     z_seq_stride=z.stride(0), y_tok_stride=y.stride(1), y_seq_stride=y.stride(0),
                     bc_tok_stride=B.stride(1), bc_seq_stride=B.stride(0), dt_seq_stride=dt_raw.stride(0))
    w = _weights(params, E, dev)
    if static_scratch:
        st = lib.ssm_prefill_host_static(ctypes.byref(dims), ctypes.byref(w), _ptr(x), _ptr(z), _ptr(B), _ptr(C),
                                         _ptr(dt_raw), _ptr(conv_cache_in), _ptr(ssm_state_in), _ptr(y),
                                         _ptr(conv_cache_out), _ptr(ssm_state_out), int(chunk_tokens), _stream(stream))
        _lib.check(st)
        return y, conv_cache_out, ssm_state_out
    ws = int(lib.ssm_prefill_host_workspace_bytes(ctypes.byref(dims), int(chunk_tokens)))
    if workspace is None or workspace.numel() < ws:
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=dev)
    st = lib.ssm_prefill_host(ctypes.byref(dims), ctypes.byref(w), _ptr(x), _ptr(z), _ptr(B), _ptr(C), _ptr(dt_raw),
                              _ptr(conv_cache_in), _ptr(ssm_state_in), _ptr(y), _ptr(conv_cache_out),
                              _ptr(ssm_state_out), _ptr(workspace), workspace.numel(), int(chunk_tokens),
                              _stream(stream))
    _lib.check(st)
    return y, conv_cache_out, ssm_state_out


def segment_summary_workspace_bytes(batch, seqlen, E, io_dtype=torch.bfloat16) -> int:
    lib = _lib.load()
    return int(lib.ssm_segment_summary_workspace_bytes(ctypes.byref(make_dims(batch, seqlen, E, io_dtype))))


def segment_summary(x, B, dt_raw, params, *, conv_cache_in=None, summary=None, workspace=None, dt_min=1e-4,
                    dt_max=1.0, discretization="euler", stream=None):
    """Summary of one segment of a sequence for the sequence-parallel prefill
    (ssm_segment_summary): x [b, T, E] (last dim contiguous), B [b, T, 16],
    dt_raw [b, T]; conv_cache_in [b, 3, E] = raw x rows before the segment, or
    None for zeros. Returns summary [b, 17, E] fp32: the zero-start final
    state in rows 0..15, the dt sum in row 16."""
    lib = _lib.load()
    b, T, E = x.shape
    dev = x.device
    for n, t in (("x", x), ("B", B), ("dt_raw", dt_raw), ("conv_cache_in", conv_cache_in), ("summary", summary),
                 ("workspace", workspace)):
        _need_cuda(n, t, dev)
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    if B.shape != (b, T, 16) or dt_raw.shape != (b, T):
        raise ValueError("shape mismatch: B [b,T,16], dt_raw [b,T]")
    if x.stride(2) != 1 or B.stride(2) != 1 or dt_raw.stride(1) != 1:
        raise ValueError("the innermost dimension of x, B, dt_raw must be contiguous")
    if conv_cache_in is not None and (conv_cache_in.shape != (b, 3, E) or conv_cache_in.dtype != x.dtype
                                      or not conv_cache_in.is_contiguous()):
        raise ValueError("conv_cache_in must be a contiguous [b, 3, E] tensor in the io dtype")
    if summary is None:
        summary = torch.empty((b, 17, E), dtype=torch.float32, device=dev)
    if summary.shape != (b, 17, E) or summary.dtype != torch.float32 or not summary.is_contiguous():
        raise ValueError("summary must be a contiguous float32 [b, 17, E] tensor")
    dims = make_dims(b, T, E, x.dtype, dt_min, dt_max, discretization, x_tok_stride=x.stride(1),
                     x_seq_stride=x.stride(0), bc_tok_stride=B.stride(1), bc_seq_stride=B.stride(0),
                     dt_seq_stride=dt_raw.stride(0))
    ws = int(lib.ssm_segment_summary_workspace_bytes(ctypes.byref(dims)))
    if workspace is None and ws:
        workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
    if ws and workspace.numel() * workspace.element_size() < ws:
        raise ValueError(f"workspace needs {ws} bytes")
    w = _weights(params, E, dev)
    st = lib.ssm_segment_summary(ctypes.byref(dims), ctypes.byref(w), _ptr(x), _ptr(B), _ptr(dt_raw),
                                 _ptr(conv_cache_in), _ptr(summary), _ptr(workspace) if ws else None, ws,
                                 _stream(stream))
    _lib.check(st)
    return summary


def segment_carry(summaries, params, *, ssm_state_in=None, out=None, stream=None):
    """State entering the segment after the summarised ones
    (ssm_segment_carry): summaries [count, b, 17, E] fp32 (count may be 0);
    ssm_state_in [b, E, 16] = the state before segment 0, or None for zeros.
    Returns [b, E, 16] fp32 (out may alias ssm_state_in)."""
    lib = _lib.load()
    count, b, rows, E = summaries.shape
    dev = summaries.device
    for n, t in (("summaries", summaries), ("ssm_state_in", ssm_state_in), ("out", out)):
        _need_cuda(n, t, dev)
    if rows != 17 or summaries.dtype != torch.float32 or not summaries.is_contiguous():
        raise ValueError("summaries must be a contiguous float32 [count, b, 17, E] tensor")
    if out is None:
        out = torch.empty((b, E, 16), dtype=torch.float32, device=dev)
    for n, t in (("ssm_state_in", ssm_state_in), ("out", out)):
        if t is not None and (t.shape != (b, E, 16) or t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{n} must be a contiguous float32 [b, E, 16] tensor")
    dims = make_dims(b, 0, E, torch.float32)
    w = _weights(params, E, dev)
    st = lib.ssm_segment_carry(ctypes.byref(dims), ctypes.byref(w), _ptr(summaries) if count else None, int(count),
                               _ptr(ssm_state_in), _ptr(out), _stream(stream))
    _lib.check(st)
    return out


PROJ_NAMES = ("W_in", "W_x", "W_out")


def make_block_dims(batch, seqlen, d_model, E, dt_min=1e-4, dt_max=1.0, discretization="euler"):
    d = _lib.SsmBlockDims()
    d.batch, d.seqlen, d.d_model, d.d_inner, d.d_state, d.d_conv = batch, seqlen, d_model, E, 16, 4
    d.dt_min, d.dt_max = dt_min, dt_max
    d.io_dtype = _lib.SSM_BF16
    d.discretization = _DISC[discretization]
    return d


def block_workspace_bytes(batch, seqlen, d_model, E) -> int:
    lib = _lib.load()
    return int(lib.ssm_block_workspace_bytes(ctypes.byref(make_block_dims(batch, seqlen, d_model, E))))


def block_forward(hidden, params, proj, *, conv_cache_in=None, ssm_state_in=None, out=None, conv_cache_out=None,
                  ssm_state_out=None, dt_min=1e-4, dt_max=1.0, discretization="euler", workspace=None, stream=None):
    """The whole block forward (ssm_block_forward): hidden [b, L, D] bf16 ->
    out [b, L, D] bf16, with proj = {"W_in": [2E, D], "W_x": [33, E],
    "W_out": [D, E]} bf16 and the core's parameters in `params`.
    Returns (out, conv_cache_out [b, 3, E], ssm_state_out [b, E, 16])."""
    lib = _lib.load()
    b, L, Dm = hidden.shape
    dev = hidden.device
    E = proj["W_x"].shape[1]
    for n, t in (("hidden", hidden), ("out", out), ("conv_cache_in", conv_cache_in), ("ssm_state_in", ssm_state_in),
                 ("conv_cache_out", conv_cache_out), ("ssm_state_out", ssm_state_out)):
        _need_cuda(n, t, dev)
    for n in PROJ_NAMES:
        _need_cuda(n, proj[n], dev)
        if proj[n].dtype != torch.bfloat16 or not proj[n].is_contiguous():
            raise ValueError(f"{n} must be a contiguous bfloat16 tensor")
    if proj["W_in"].shape != (2 * E, Dm) or proj["W_x"].shape != (33, E) or proj["W_out"].shape != (Dm, E):
        raise ValueError("W_in must be [2E, D], W_x [33, E] and W_out [D, E]")
    if hidden.dtype != torch.bfloat16 or not hidden.is_contiguous():
        raise ValueError("hidden must be a contiguous bfloat16 tensor")
    if out is None:
        out = torch.empty((b, L, Dm), dtype=torch.bfloat16, device=dev)
    if conv_cache_out is None:
        conv_cache_out = torch.empty((b, 3, E), dtype=torch.bfloat16, device=dev)
    if ssm_state_out is None:
        ssm_state_out = torch.empty((b, E, 16), dtype=torch.float32, device=dev)
    dims = make_block_dims(b, L, Dm, E, dt_min, dt_max, discretization)
    w = _weights(params, E, dev)
    pw = _lib.SsmBlockWeights(proj["W_in"].data_ptr(), proj["W_x"].data_ptr(), proj["W_out"].data_ptr())
    ws = int(lib.ssm_block_workspace_bytes(ctypes.byref(dims)))
    if workspace is None or workspace.numel() < ws:
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=dev)
    st = lib.ssm_block_forward(ctypes.byref(dims), ctypes.byref(w), ctypes.byref(pw), _ptr(hidden),
                               _ptr(conv_cache_in), _ptr(ssm_state_in), _ptr(out), _ptr(conv_cache_out),
                               _ptr(ssm_state_out), _ptr(workspace), workspace.numel(), _stream(stream))
    _lib.check(st)
    return out, conv_cache_out, ssm_state_out


def proj_gemm_workspace_bytes(M, N, K) -> int:
    lib = _lib.load()
    return int(lib.ssm_proj_gemm_workspace_bytes(int(M), int(N), int(K)))


def proj_gemm(A, W, *, out=None, workspace=None, stream=None):
    """One projection of the block (ssm_proj_gemm): out = A @ W^T with A [M, K]
    and W [N, K] contiguous bf16 CUDA tensors; returns out [M, N] bf16. The
    cut-tile scratch, when the shape needs one, is `workspace` or allocated."""
    lib = _lib.load()
    M, K = A.shape
    N = W.shape[0]
    dev = A.device
    for n, t in (("A", A), ("W", W), ("out", out)):
        _need_cuda(n, t, dev)
        if t is not None and (t.dtype != torch.bfloat16 or not t.is_contiguous()):
            raise ValueError(f"{n} must be a contiguous bfloat16 tensor")
    if W.shape[1] != K:
        raise ValueError("A [M, K] and W [N, K] must share K")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if out.shape != (M, N):
        raise ValueError("out must be [M, N]")
    ws = int(lib.ssm_proj_gemm_workspace_bytes(M, N, K))
    if ws and (workspace is None or workspace.numel() * workspace.element_size() < ws):
        workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
    _lib.check(lib.ssm_proj_gemm(_ptr(A), _ptr(W), _ptr(out), M, N, K, _ptr(workspace) if ws else None, ws,
                                 _stream(stream)))
    return out


def ssd_chunk_scan(cb, x, dt, dA_cumsum, C, prev_states, D=None, *, out=None, stream=None):
    """Mamba-2 chunk-scan output (ssm_ssd_chunk_scan). cb [b, nc, G, cs, cs],
    x [b, L, H, P], C [b, L, G, N], prev_states [b, nc, H, P, N]: bf16;
    dt, dA_cumsum [b, H, nc, cs] and D [H]: fp32. Returns out [b, L, H, P] bf16."""
    lib = _lib.load()
    b, L, H, P = x.shape
    _, nc, G, cs, _ = cb.shape
    N = C.shape[-1]
    dev = x.device
    for n, t in (("cb", cb), ("x", x), ("dt", dt), ("dA_cumsum", dA_cumsum), ("C", C), ("prev_states", prev_states),
                 ("D", D), ("out", out)):
        _need_cuda(n, t, dev)
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for n, t in (("cb", cb), ("x", x), ("C", C), ("prev_states", prev_states)):
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{n} must be bfloat16")
    for n, t in (("dt", dt), ("dA_cumsum", dA_cumsum), ("D", D)):
        if t is not None and t.dtype != torch.float32:
            raise ValueError(f"{n} must be float32")
    if (cb.shape != (b, nc, G, cs, cs) or C.shape != (b, L, G, N) or prev_states.shape != (b, nc, H, P, N)
            or dt.shape != (b, H, nc, cs) or dA_cumsum.shape != dt.shape or (D is not None and D.shape != (H,))):
        raise ValueError("shape mismatch between the chunk-scan operands")
    if out is None:
        out = torch.empty_like(x)
    d = _lib.SsmSsdDims(b, L, H, P, G, N, cs)
    st = lib.ssm_ssd_chunk_scan(ctypes.byref(d), _ptr(cb), _ptr(x), _ptr(dt), _ptr(dA_cumsum), _ptr(C),
                                _ptr(prev_states), _ptr(D), _ptr(out), _stream(stream))
    _lib.check(st)
    return out


try:  # the current stream's handle without a Stream object (3 us of a small call)
    from torch._C import _cuda_getCurrentRawStream as _current_raw_stream
except ImportError:
    def _current_raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _raw_stream(device, stream):
    """Handle of the call's stream on device number `device`, which must be the current one: kernels are launched
    there."""
    if device != torch.cuda.current_device():
        raise RuntimeError(f"tensors are on cuda:{device}, but the current device is "
                           f"cuda:{torch.cuda.current_device()}: make the call under torch.cuda.device(...)")
    if stream is None:
        return _current_raw_stream(device)
    if stream.device_index != device:
        raise RuntimeError(f"tensors are on cuda:{device}, but the stream is on cuda:{stream.device_index}")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A buffer of the call, allocated on its stream: once dropped, its memory goes to later work of that stream."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(t, stream):
    """The same for a dense buffer of t's shape and type (half the host time of torch.empty)."""
    if stream is None or not t.is_cuda:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        return torch.empty_like(t, memory_format=torch.contiguous_format)


def _workspace(workspace, nbytes, device, stream):
    """The caller's workspace where it is large enough, else a new one."""
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        return _empty(nbytes, torch.uint8, device, stream)
    return workspace


def _address(t):
    return None if t is None else t.data_ptr()


def _one_device(names, *tensors):
    """Device number that the tensors (or None) share; the first must be a tensor. names: theirs, in one string."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != device or device < 0):
            for name, t in zip(names.split(), tensors):
                _need_cuda(name, t, tensors[0].device)
    return device


def _stride(name, t, i):
    """t's stride along dimension i for the C call: 0 (the dense default) where there is one index or none; an
    expanded dimension has no stride that the call could express."""
    if t.shape[i] <= 1 or not t.numel():
        return 0
    s = t.stride(i)
    if s == 0:
        raise ValueError(f"{name} is expanded along dimension {i}: make it contiguous")
    return s


def _row_stride(name, t):
    """The one stride between the rows of t [rows, dim] or [b, L, dim]."""
    if t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError(f"the rows of {name} must be contiguous")
    if t.dim() == 2:
        return _stride(name, t, 0)
    s0, s1 = _stride(name, t, 0), _stride(name, t, 1)
    if s0 and s1 and s0 != t.shape[1] * s1:
        raise ValueError(f"the rows of {name} must be at one stride")
    return s1 or s0


def _dense_heads(name, t):
    """The last two dimensions (head, channel) dense."""
    sh, st = t.shape, t.stride()
    if ((sh[-1] > 1 and st[-1] != 1) or (sh[-2] > 1 and st[-2] != sh[-1])) and t.numel():
        raise ValueError(f"the head and channel dimensions of {name} must be contiguous")


def _delta_strides(name, t, tokens, sequences, heads=True):
    """t's token and sequence strides for the C call (see _stride; dimension None: 0); with `heads`, its last two
    dimensions (head, channel) must be dense."""
    if not t.numel():
        return 0, 0
    if heads and not t.is_contiguous():
        _dense_heads(name, t)
    sh, st = t.shape, t.stride()
    a = 0 if tokens is None or sh[tokens] <= 1 else st[tokens] or _stride(name, t, tokens)
    b = 0 if sequences is None or sh[sequences] <= 1 else st[sequences] or _stride(name, t, sequences)
    return a, b


def _delta_dims(q, k, v, g, beta, out, scale, qk_l2norm, batch, seqlen, tokens, sequences):
    """Checks the token tensors of the delta rule ([..., heads, channels]; g, beta [..., heads]) and fills
    SsmDeltaDims; tokens, sequences: the dimensions that hold them, or None."""
    qs, vs, bf16 = q.shape, v.shape, torch.bfloat16
    lead, G, H = qs[:-2], qs[-2], vs[-2]
    if q.dtype is not bf16 or k.dtype is not bf16 or v.dtype is not bf16 or out.dtype is not bf16:
        raise ValueError("q, k, v and out must be bfloat16")
    if k.shape != qs or vs[:-2] != lead or G == 0 or H % G:
        raise ValueError("k must have q's shape, v its tokens, and v's heads must be a multiple of q's")
    if out.shape != vs:
        raise ValueError("out must have v's shape")
    if g.dtype is not torch.float32 or beta.dtype is not torch.float32 or g.shape != vs[:-1] or beta.shape != vs[:-1]:
        raise ValueError("g and beta must be float32 with one value per token and head of v")
    if scale is None:
        scale = 0.0
    elif not 1e-45 < scale <= 3.4028234663852886e38:  # 0 in the dims is the default
        raise ValueError("scale must be positive and finite in float32")
    if q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous() and g.is_contiguous() \
            and beta.is_contiguous():
        strides = ()
    else:
        if H > 1 and g.numel() and (g.stride(-1) != 1 or beta.stride(-1) != 1):
            raise ValueError("the heads of g and beta must be contiguous")
        gs = _delta_strides("g", g, tokens, sequences, False)
        if _delta_strides("beta", beta, tokens, sequences, False) != gs:
            raise ValueError("g and beta must share strides")
        strides = (*_delta_strides("q", q, tokens, sequences), *_delta_strides("k", k, tokens, sequences),
                   *_delta_strides("v", v, tokens, sequences), *_delta_strides("out", out, tokens, sequences), *gs)
    return _lib.SsmDeltaDims(batch, seqlen, H, G, qs[-1], vs[-1], scale, 1 if qk_l2norm else 0, *strides)


def _delta_state(name, t, n, H, dv, dk):
    if t.dtype is not torch.float32 or t.shape != (n, H, dv, dk) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 [{n}, {H}, {dv}, {dk}] tensor")


def delta_prefill_workspace_bytes(batch, seqlen, nheads, ngroups, d_key, d_value, packed=False) -> int:
    """Workspace bytes of `delta_prefill`; with packed, for `batch` sequences in a buffer of `seqlen` tokens."""
    d = _lib.SsmDeltaDims(batch, seqlen, nheads, ngroups, d_key, d_value)
    return int(_lib.load().ssm_delta_prefill_workspace_bytes(ctypes.byref(d), int(bool(packed))))


def delta_prefill(q, k, v, g, beta, *, state_in=None, cu_seqlens=None, scale=None, qk_l2norm=False, out=None,
                  state_out=None, workspace=None, stream=None):
    """Gated delta rule over whole sequences (ssm_delta_prefill): per head
    S <- a S + beta (v - a S k) k^T with a = exp(g), out = scale S q. q, k
    [b, L, G, dk], v [b, L, H, dv] bf16 (head h reads group h // (H // G)), g,
    beta [b, L, H] fp32; the last two dimensions dense, token and sequence
    strides as they are. With cu_seqlens (int32 [n + 1] on the device) the
    tensors are packed, [T, ...], sequence i being rows cu_seqlens[i] to
    cu_seqlens[i + 1]; rows of no sequence keep what `out` held. state_in
    [n, H, dv, dk] fp32 or None = zeros; scale None = dk ** -0.5; qk_l2norm
    normalises q and k inside. Returns (out, state_out)."""
    lib = _lib.load()
    packed = cu_seqlens is not None
    if q.dim() != (3 if packed else 4) or v.dim() != q.dim():
        raise ValueError("q must be [b, L, G, dk] and v [b, L, H, dv], or [tokens, ...] with cu_seqlens")
    if out is None:
        out = _empty_like(v, stream)
    dev = _one_device("q k v g beta out state_in state_out cu_seqlens workspace", q, k, v, g, beta, out, state_in,
                      state_out, cu_seqlens, workspace)
    if packed:
        if cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() \
                or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a contiguous int32 [sequences + 1] tensor")
        n = cu_seqlens.numel() - 1
        d = _delta_dims(q, k, v, g, beta, out, scale, qk_l2norm, n, q.shape[0], 0, None)
    else:
        n = q.shape[0]
        d = _delta_dims(q, k, v, g, beta, out, scale, qk_l2norm, n, q.shape[1], 1, 0)
    H, dv, dk = v.shape[-2], v.shape[-1], q.shape[-1]
    if state_in is not None:
        _delta_state("state_in", state_in, n, H, dv, dk)
    if state_out is None:
        state_out = _empty((n, H, dv, dk), torch.float32, q.device, stream) if state_in is None \
            else _empty_like(state_in, stream)
    else:
        _delta_state("state_out", state_out, n, H, dv, dk)
    ref = ctypes.byref(d)
    ws = lib.ssm_delta_prefill_workspace_bytes(ref, 1 if packed else 0)
    if ws:
        workspace = _workspace(workspace, ws, q.device, stream)
    st = lib.ssm_delta_prefill(ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                               _address(cu_seqlens), _address(state_in), out.data_ptr(), state_out.data_ptr(),
                               workspace.data_ptr() if ws else None, ws, _raw_stream(dev, stream))
    _lib.check(st)
    return out, state_out


def delta_decode_step(q, k, v, g, beta, state, *, state_index=None, scale=None, qk_l2norm=False, out=None,
                      state_out=None, stream=None):
    """Gated delta rule over one token per sequence (ssm_delta_decode_step):
    q, k [b, G, dk], v [b, H, dv] bf16, g, beta [b, H] fp32. `state`
    [states, H, dv, dk] fp32 is updated in place, or read only where state_out
    (another pool of its shape) is given. state_index (int32 [b]): the state of
    each row, negative = padding, whose output and state are left alone; no two
    rows may name the same state. Returns out [b, H, dv]."""
    lib = _lib.load()
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q must be [b, G, dk] and v [b, H, dv]")
    if out is None:
        out = _empty_like(v, stream)
    if state_out is None:
        state_out = state
    dev = _one_device("q k v g beta state out state_out state_index", q, k, v, g, beta, state, out, state_out,
                      state_index)
    b, n = q.shape[0], state.shape[0]
    d = _delta_dims(q, k, v, g, beta, out, scale, qk_l2norm, b, 1, None, 0)
    if state_index is None:
        n = b
    elif state_index.dtype is not torch.int32 or state_index.shape != (b,) or not state_index.is_contiguous():
        raise ValueError("state_index must be a contiguous int32 [b] tensor")
    _delta_state("state", state, n, v.shape[1], v.shape[2], q.shape[2])
    if state_out is not state:
        _delta_state("state_out", state_out, n, v.shape[1], v.shape[2], q.shape[2])
    st = lib.ssm_delta_decode_step(ctypes.byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                                   beta.data_ptr(), _address(state_index), n, state.data_ptr(), out.data_ptr(),
                                   state_out.data_ptr(), _raw_stream(dev, stream))
    _lib.check(st)
    return out


def gated_norm(x, z, weight, *, group_size=None, eps=1e-5, gate_first=False, out=None, stream=None):
    """The norm between a scan and out_proj, fused with its gate
    (ssm_gated_norm): per group of group_size channels (None = the row),
    x / rms(x) * weight * SiLU(z), or with gate_first t / rms(t) * weight with
    t = x * SiLU(z). x, z [rows, dim] or [b, L, dim] (bf16 or fp32, last
    dimension contiguous, other strides as they are), z None = no gate; weight
    fp32 [dim], or [group_size] for every group alike. out may be x or z.
    Returns out."""
    lib = _lib.load()
    shape = x.shape
    n = len(shape)
    if (n != 2 and n != 3) or x.dtype not in _DTYPES:
        raise ValueError("x must be a float32 or bfloat16 [rows, dim] or [b, L, dim] tensor")
    dim = shape[-1]
    group = dim if group_size is None else int(group_size)
    if out is None:
        out = _empty_like(x, stream)
    dev = _one_device("x z out weight", x, z, out, weight)
    strides = []
    for name, t in (("x", x), ("z", z), ("out", out)):
        if t is None:
            strides += (0, 0)
            continue
        if t.shape == shape and t.dtype is x.dtype and t.is_contiguous():
            strides += (0, 0)
            continue
        if t.shape != shape or t.dtype is not x.dtype or (t.stride(-1) != 1 and dim > 1 and t.numel()):
            raise ValueError(f"{name} must have x's shape and dtype and a contiguous last dimension")
        strides.append(_stride(name, t, n - 2))
        strides.append(_stride(name, t, 0) if n == 3 else 0)
    ws = weight.shape
    if weight.dtype is not torch.float32 or len(ws) != 1 or ws[0] not in (dim, group) or not weight.is_contiguous():
        raise ValueError("weight must be contiguous float32 [dim] or [group_size]")
    d = _lib.SsmGatedNormDims(1 if n == 2 else shape[0], shape[n - 2], dim, group, eps, _DTYPES[x.dtype],
                              1 if gate_first else 0, 0 if ws[0] == dim else 1, *strides)
    st = lib.ssm_gated_norm(ctypes.byref(d), x.data_ptr(), _address(z), weight.data_ptr(), out.data_ptr(),
                            _raw_stream(dev, stream))
    _lib.check(st)
    return out


def residual_norm(x, residual, weight, *, post_weight=None, residual_scale=1.0, eps=1e-5, out=None,
                  residual_out=None, residual_dtype=None, stream=None):
    """The step between two blocks in one pass (ssm_residual_norm): with
    t = x, or x / rms(x) * post_weight, r = residual + residual_scale * t and
    out = r / rms(r) * weight. x [rows, dim] or [b, L, dim] (bf16 or fp32, rows
    at one stride), residual of x's shape (bf16 or fp32) or None = zeros (the
    first block; residual_dtype then picks r's type, default x's); weights fp32
    [dim]. residual_out may be residual. Returns (out, residual_out)."""
    lib = _lib.load()
    shape, dt = x.shape, x.dtype
    if len(shape) not in (2, 3) or dt not in _DTYPES:
        raise ValueError("x must be a float32 or bfloat16 [rows, dim] or [b, L, dim] tensor")
    dim = shape[-1]
    if residual is not None:
        rdt = residual.dtype
    else:
        rdt = residual_dtype or (residual_out.dtype if residual_out is not None else dt)
    if rdt not in _DTYPES or (residual_dtype is not None and residual_dtype != rdt):
        raise ValueError("the residual must be float32 or bfloat16, of residual_dtype where that is given")
    if out is None:
        out = _empty_like(x, stream)
    if residual_out is None:
        residual_out = _empty_like(residual, stream) if residual is not None and residual.shape == shape \
            else _empty(shape, rdt, x.device, stream)
    dev = _one_device("x residual out residual_out weight post_weight", x, residual, out, residual_out, weight,
                      post_weight)
    strides = []
    for name, t, want in (("x", x, dt), ("residual", residual, rdt), ("out", out, dt),
                          ("residual_out", residual_out, rdt)):
        if t is None:
            strides.append(0)
            continue
        if t.shape != shape or t.dtype is not want:
            raise ValueError(f"{name} must be a {want} tensor of x's shape")
        strides.append(0 if t.is_contiguous() else _row_stride(name, t))
    for name, t in (("weight", weight), ("post_weight", post_weight)):
        if t is not None and (t.dtype is not torch.float32 or t.shape != (dim,) or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous float32 [dim]")
    d = _lib.SsmResidualNormDims(x.numel() // max(dim, 1), dim, eps, residual_scale, _DTYPES[dt], _DTYPES[rdt],
                                 *strides)
    st = lib.ssm_residual_norm(ctypes.byref(d), x.data_ptr(), _address(residual), weight.data_ptr(),
                               _address(post_weight), out.data_ptr(), residual_out.data_ptr(),
                               _raw_stream(dev, stream))
    _lib.check(st)
    return out, residual_out


def residual_block_workspace_bytes(batch, seqlen, d_model, E) -> int:
    lib = _lib.load()
    return int(lib.ssm_residual_block_workspace_bytes(ctypes.byref(make_block_dims(batch, seqlen, d_model, E))))


def residual_block_forward(x, residual, params, proj, norm_weight, *, post_weight=None, residual_scale=1.0, eps=1e-5,
                           residual_dtype=torch.float32, residual_out=None, conv_cache_in=None, ssm_state_in=None,
                           out=None, conv_cache_out=None, ssm_state_out=None, dt_min=1e-4, dt_max=1.0,
                           discretization="euler", workspace=None, stream=None):
    """One pre-norm residual layer around the block (ssm_residual_block_forward):
    (hidden, r) = residual_norm(x, residual, norm_weight, ...), out =
    block_forward(hidden). x [b, L, D] bf16 is the previous block's output (or
    the embedding, with residual None), contiguous; residual and r [b, L, D] in
    residual_dtype, contiguous. The next layer takes (out, r). Returns (out, r,
    conv_cache_out, ssm_state_out)."""
    lib = _lib.load()
    b, L, Dm = x.shape
    dev = x.device
    E = proj["W_x"].shape[1]
    if residual is not None:
        residual_dtype = residual.dtype
    if residual_dtype not in _DTYPES:
        raise ValueError("the residual must be float32 or bfloat16")
    if residual_out is None:
        residual_out = _empty((b, L, Dm), residual_dtype, dev, stream)
    if out is None:
        out = _empty((b, L, Dm), torch.bfloat16, dev, stream)
    if conv_cache_out is None:
        conv_cache_out = _empty((b, 3, E), torch.bfloat16, dev, stream)
    if ssm_state_out is None:
        ssm_state_out = _empty((b, E, 16), torch.float32, dev, stream)
    full, cache, state = (b, L, Dm), (b, 3, E), (b, E, 16)
    for n, t, shape, dt in (("x", x, full, torch.bfloat16), ("residual", residual, full, residual_dtype),
                            ("residual_out", residual_out, full, residual_dtype), ("out", out, full, torch.bfloat16),
                            ("W_in", proj["W_in"], (2 * E, Dm), torch.bfloat16),
                            ("W_x", proj["W_x"], (33, E), torch.bfloat16),
                            ("W_out", proj["W_out"], (Dm, E), torch.bfloat16),
                            ("norm_weight", norm_weight, (Dm,), torch.float32),
                            ("post_weight", post_weight, (Dm,), torch.float32),
                            ("conv_cache_in", conv_cache_in, cache, torch.bfloat16),
                            ("conv_cache_out", conv_cache_out, cache, torch.bfloat16),
                            ("ssm_state_in", ssm_state_in, state, torch.float32),
                            ("ssm_state_out", ssm_state_out, state, torch.float32)):
        _need_cuda(n, t, dev)
        if t is not None and (t.shape != shape or t.dtype != dt or not t.is_contiguous()):
            raise ValueError(f"{n} must be a contiguous {dt} tensor of shape {shape}")
    dims = make_block_dims(b, L, Dm, E, dt_min, dt_max, discretization)
    w = _weights(params, E, dev)
    pw = _lib.SsmBlockWeights(proj["W_in"].data_ptr(), proj["W_x"].data_ptr(), proj["W_out"].data_ptr())
    nw = _lib.SsmBlockNorm(norm_weight.data_ptr(), None if post_weight is None else post_weight.data_ptr(), eps,
                           residual_scale, _DTYPES[residual_dtype])
    ws = int(lib.ssm_residual_block_workspace_bytes(ctypes.byref(dims)))
    workspace = _workspace(workspace, max(ws, 1), dev, stream)
    _need_cuda("workspace", workspace, dev)
    _lib.check(lib.ssm_residual_block_forward(
        ctypes.byref(dims), ctypes.byref(w), ctypes.byref(pw), ctypes.byref(nw), _ptr(x), _ptr(residual),
        _ptr(conv_cache_in), _ptr(ssm_state_in), _ptr(residual_out), _ptr(out), _ptr(conv_cache_out),
        _ptr(ssm_state_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _raw_stream(x.get_device(), stream)))
    return out, residual_out, conv_cache_out, ssm_state_out


def decode_step(x, z, B, C, dt_raw, params, conv_cache, ssm_state, *, y=None, dt_min=1e-4, dt_max=1.0,
                discretization="euler", stream=None):
    """One-token block core. x, z: [b, E] (last dim contiguous); B, C: [b, 16];
    dt_raw: [b]; conv_cache [b, 3, E] and ssm_state [b, E, 16] are updated in
    place. Returns y [b, E]."""
    lib = _lib.load()
    b, E = x.shape
    dev = x.device
    for n, t in (("x", x), ("z", z), ("B", B), ("C", C), ("dt_raw", dt_raw), ("conv_cache", conv_cache),
                 ("ssm_state", ssm_state), ("y", y)):
        _need_cuda(n, t, dev)
    if x.dtype not in _DTYPES or z.dtype != x.dtype or conv_cache.dtype != x.dtype:
        raise ValueError("x, z and conv_cache must share an io dtype")
    if z.shape != (b, E) or B.shape != (b, 16) or C.shape != (b, 16) or dt_raw.shape != (b,):
        raise ValueError("shape mismatch: z [b,E], B/C [b,16], dt_raw [b]")
    if x.stride(1) != 1 or z.stride(1) != 1 or B.stride(1) != 1 or B.stride() != C.stride():
        raise ValueError("innermost dims must be contiguous and B, C share strides")
    if conv_cache.shape != (b, 3, E) or not conv_cache.is_contiguous():
        raise ValueError("conv_cache must be a contiguous [b, 3, E] tensor")
    if ssm_state.shape != (b, E, 16) or ssm_state.dtype != torch.float32 or not ssm_state.is_contiguous():
        raise ValueError("ssm_state must be a contiguous float32 [b, E, 16] tensor")
    if y is None:
        y = torch.empty((b, E), dtype=x.dtype, device=dev)
    dims = make_dims(b, 1, E, x.dtype, dt_min, dt_max, discretization, x_seq_stride=x.stride(0),
                     z_seq_stride=z.stride(0), y_seq_stride=y.stride(0), bc_seq_stride=B.stride(0),
                     dt_seq_stride=dt_raw.stride(0))
    w = _weights(params, E, dev)
    st = lib.ssm_decode_step(ctypes.byref(dims), ctypes.byref(w), _ptr(x), _ptr(z), _ptr(B), _ptr(C), _ptr(dt_raw),
                             _ptr(y), _ptr(conv_cache), _ptr(ssm_state), _stream(stream))
    _lib.check(st)
    return y


def check_device_error(stream=None):
    """ssm_check_device_error: synchronises `stream`, then raises SsmError
    (status SSM_ERR_DEVICE) if a kernel's bounded wait gave up since the last
    check, clearing the device error word."""
    lib = _lib.load()
    _lib.check(lib.ssm_check_device_error(_stream(stream)))


def selftest_bounded_wait(limit_ns=1_000_000, stream=None):
    """ssm_selftest_bounded_wait: a kernel whose wait can never complete gives
    up after limit_ns and reports through the device error word."""
    lib = _lib.load()
    _lib.check(lib.ssm_selftest_bounded_wait(int(limit_ns), _stream(stream)))
