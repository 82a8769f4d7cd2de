"""Python binding of libkda.so, the MI355X (gfx950) KDA chunked-prefill forward.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in include/kda.h.  Tensors are torch tensors
used as device memory; the stream defaults to torch's current stream.  There
is no CPU fallback: if libkda.so is missing, every call raises.

    ws = torch.zeros(kda_get_workspace_size(T, H, N), dtype=torch.uint8, device="cuda")
    kda_chunk_prefill_fwd(q, k, v, g, beta_logits, A_log, dt_bias, lower_bound, scale,
                          initial_state, cu_seqlens, out, final_state, ws)

q, k, v, g, out and beta_logits may be strided views (channels contiguous, for
[T, H, 128] both strides multiples of 8 elements): they then go through
kda_chunk_prefill_fwd_strided, with no copy.

The operators around the forward (include/kda_layer.h) are here too:

    kda_add_rms_norm(x, residual, weight, 1e-6, hidden)
    kda_w4_proj(hidden, w, scales, None, qkvab, 128)
    kda_gdr_decode_step(q, k, v, a, beta_logits, A_log, dt_bias, scale, pool, slots, out)

and those on microscaled 4-bit numbers (include/kda_mx4.h):

    kda_mx4_quant(x, codes, scales)
    kda_mx4_proj(codes, scales, w, w_scales, y)       # or (x, None, w, w_scales, y) for few rows
    kda_mx4_moe(hidden, router, bias, w_up, s_up, w_down, s_down, out, ids, gates, ws)
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

__all__ = ["kda_get_workspace_size", "kda_chunk_prefill_fwd", "kda_status_string",
           "kda_workspace_status",
           "kda_last_hip_error", "kda_debug_set_vsplit", "kda_debug_set_kernel", "kda_debug_set_segment", "kda_debug_segment_length", "kda_debug_two_workgroups", "kda_spec_decode_step", "kda_chunk_prefill_fwd_noalloc", "kda_gate_proj",
           "kda_gate_proj_workspace_size", "kda_gdr_get_workspace_size", "kda_gdr_prefill_fwd",
           "kda_gdr_decode_step", "kda_add_rms_norm", "kda_w4_proj", "kda_mx4_quant", "kda_mx4_dequant",
           "kda_mx4_proj", "kda_mx4_moe_workspace_size", "kda_mx4_moe", "KdaError", "library_path", "load_library"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libkda.so")

HEAD_DIM = 128
KDA_OK = 0
KDA_STATE_FP32 = 0
KDA_STATE_BF16 = 1

_lib = None


class _Strides(ctypes.Structure):
    """kda_strides_t of include/kda.h (element strides)."""
    _fields_ = [(n, ctypes.c_int64) for n in (
        "q_token", "q_head", "k_token", "k_head", "v_token", "v_head", "g_token", "g_head",
        "beta_token", "beta_head", "out_token", "out_head")]


class _GdrStrides(ctypes.Structure):
    """kda_gdr_strides_t of include/kda_layer.h (element strides)."""
    _fields_ = [(n, ctypes.c_int64) for n in (
        "q_token", "q_head", "k_token", "k_head", "v_token", "v_head", "a_token", "a_head",
        "beta_token", "beta_head", "out_token", "out_head")]


class KdaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libkda.so once; raises if it has not been built.

    torch's wheel carries its own HIP runtime (libamdhip64, SONAME
    libamdhip64.so.7, the same SONAME as the system ROCm copy).  torch is
    imported first so that its runtime is in the process before libkda.so is
    mapped: the dynamic loader then resolves libkda.so's libamdhip64.so.7 to
    that same copy.  Loading libkda.so first would bring in the system copy, and
    torch would then load a second HIP runtime that sees no device.
    """
    global _lib
    if _lib is None:
        try:
            import torch  # noqa: F401  (see above: one HIP runtime per process)
        except ImportError:
            pass
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with "
                "`python -m gated_delta_rule_tok_amd.build` (there is no fallback path)")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I32, I64, SZ, F = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                              ctypes.c_float)
        lib.kda_get_workspace_size.argtypes = [I64, I32, I32]
        lib.kda_get_workspace_size.restype = SZ
        lib.kda_chunk_prefill_fwd.argtypes = [P, P, P, P, P, P, P, F, F, P, P, P, P, P, P,
                                              I64, I32, I32, ctypes.c_int, SZ]
        lib.kda_chunk_prefill_fwd.restype = ctypes.c_int
        lib.kda_chunk_prefill_fwd_strided.argtypes = [P, P, P, P, P, P, P, F, F, P, P, P, P, P,
                                                      P, I64, I32, I32, ctypes.c_int, SZ,
                                                      ctypes.POINTER(_Strides)]
        lib.kda_chunk_prefill_fwd_strided.restype = ctypes.c_int
        lib.kda_chunk_prefill_fwd_checkpoints.argtypes = [
            P, P, P, P, P, P, P, F, F, P, P, P, P, P, P, I64, I32, I32, ctypes.c_int, SZ,
            ctypes.POINTER(_Strides), P, I32, I64]
        lib.kda_chunk_prefill_fwd_checkpoints.restype = ctypes.c_int
        lib.kda_chunk_prefill_fwd_noalloc.argtypes = [P, P, P, P, P, P, P, F, F, P, P, P, P, P, P,
                                                      I64, I32, I32, ctypes.c_int]
        lib.kda_chunk_prefill_fwd_noalloc.restype = ctypes.c_int
        lib.kda_gate_proj_workspace_size.argtypes = [I32, I32, I32]
        lib.kda_gate_proj_workspace_size.restype = SZ
        lib.kda_gate_proj.argtypes = [P, P, P, P, P, P, SZ, P, I32, I32, I32, I32]
        lib.kda_gate_proj.restype = ctypes.c_int
        lib.kda_spec_decode_step.argtypes = [P, P, P, P, P, P, P, F, F, P, I64, P, P, I32, P, P,
                                             P, P, I64, I32, I32, ctypes.c_int, SZ]
        lib.kda_spec_decode_step.restype = ctypes.c_int
        lib.kda_gdr_get_workspace_size.argtypes = [I64, I32, I32, I32]
        lib.kda_gdr_get_workspace_size.restype = SZ
        lib.kda_gdr_prefill_fwd.argtypes = [P, P, P, P, P, P, P, F, P, P, P, P, P, P, I64, I32, I32,
                                            I32, ctypes.c_int, SZ, ctypes.POINTER(_GdrStrides)]
        lib.kda_gdr_prefill_fwd.restype = ctypes.c_int
        lib.kda_gdr_decode_step.argtypes = [P, P, P, P, P, P, P, F, P, I64, P, P, P, I32, I32, I32,
                                            ctypes.c_int, ctypes.POINTER(_GdrStrides)]
        lib.kda_gdr_decode_step.restype = ctypes.c_int
        lib.kda_add_rms_norm.argtypes = [P, P, P, F, P, P, P, I64, I32, I64, I64, I64, ctypes.c_int,
                                         I32]
        lib.kda_add_rms_norm.restype = ctypes.c_int
        lib.kda_w4_proj.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I64, I64]
        lib.kda_w4_proj.restype = ctypes.c_int
        lib.kda_mx4_quant.argtypes = [P, P, P, P, I64, I32, I64]
        lib.kda_mx4_quant.restype = ctypes.c_int
        lib.kda_mx4_dequant.argtypes = [P, P, P, P, I64, I32, I64]
        lib.kda_mx4_dequant.restype = ctypes.c_int
        lib.kda_mx4_proj.argtypes = [P, P, P, P, P, P, I64, I32, I32, I64, I64]
        lib.kda_mx4_proj.restype = ctypes.c_int
        lib.kda_mx4_moe_workspace_size.argtypes = [I32, I32, I32, I32, I32, I32]
        lib.kda_mx4_moe_workspace_size.restype = SZ
        lib.kda_mx4_moe.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I64,
                                    I64, ctypes.c_int, I32, F, SZ]
        lib.kda_mx4_moe.restype = ctypes.c_int
        lib.kda_status_string.argtypes = [ctypes.c_int]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_last_hip_error.argtypes = []
        lib.kda_last_hip_error.restype = ctypes.c_char_p
        lib.kda_debug_set_kernel.argtypes = [ctypes.c_int]
        lib.kda_debug_set_kernel.restype = ctypes.c_int
        lib.kda_debug_set_vsplit.argtypes = [ctypes.c_int]
        lib.kda_debug_set_vsplit.restype = ctypes.c_int
        lib.kda_debug_set_segment.argtypes = [ctypes.c_int]
        lib.kda_debug_set_segment.restype = ctypes.c_int
        lib.kda_debug_segment_length.argtypes = [I64, I32, I32]
        lib.kda_debug_segment_length.restype = I32
        lib.kda_debug_two_workgroups.argtypes = [I64, I32, I32, I32]
        lib.kda_debug_two_workgroups.restype = I32
        _lib = lib
    return _lib


def kda_get_workspace_size(max_tokens: int, heads: int, max_seqs: int) -> int:
    return int(load_library().kda_get_workspace_size(int(max_tokens), int(heads), int(max_seqs)))


def kda_workspace_status(workspace) -> int:
    """The workspace's status word (its first 4 bytes, see include/kda.h): 0 while
    every call that used it ran to completion normally; nonzero (the kind of
    wait, 1: LDS counters) once a kernel gave up a bounded wait (the outputs of
    that call are void).  Synchronises the device."""
    import torch
    return int(workspace[:4].view(torch.int32)[0].item())


def kda_status_string(status: int) -> str:
    return load_library().kda_status_string(int(status)).decode()


def kda_last_hip_error() -> str:
    return load_library().kda_last_hip_error().decode()


def kda_debug_set_kernel(k: int) -> int:
    """Test hook: 0 automatic (default), 1 64-token kernel, 2 token-serial
    kernel, 3 token-serial kernel with decode staging, 4 pipelined 16-token
    kernel (where it applies), 5 pipelined 32-token kernel."""
    prev = load_library().kda_debug_set_kernel(int(k))
    if prev < 0:
        raise ValueError(f"invalid kernel selector {k}")
    return prev


def kda_debug_set_vsplit(s: int) -> int:
    """Test hook: force the value split (1, 2, 4, 8) or 0 for automatic."""
    prev = load_library().kda_debug_set_vsplit(int(s))
    if prev < 0:
        raise ValueError(f"invalid value split {s}")
    return prev


def kda_debug_set_segment(length: int) -> int:
    """Test hook: the segment-parallel schedule -- 0 automatic, 1 never, or
    segments of `length` tokens (a multiple of 16) where the call allows it."""
    prev = load_library().kda_debug_set_segment(int(length))
    if prev < 0:
        raise ValueError(f"invalid segment length {length}")
    return prev


def kda_debug_segment_length(num_tokens: int, heads: int, num_seqs: int) -> int:
    """The segment length a call of these sizes would use (0: one piece)."""
    return int(load_library().kda_debug_segment_length(int(num_tokens), int(heads), int(num_seqs)))


def kda_debug_two_workgroups(num_tokens: int, heads: int, num_seqs: int, cus: int = 256) -> bool:
    """Whether a call of these sizes (with the workspace's second part) runs
    the 16-token kernel in two workgroups per (sequence, head) on a device of
    cus compute units."""
    return bool(load_library().kda_debug_two_workgroups(int(num_tokens), int(heads), int(num_seqs),
                                                        int(cus)))


def _check(t, name, dtype, shape=None, strided=False):
    """Device pointer of t after the dtype/shape checks.  strided: the leading
    two strides may be anything non-negative (the last dim must be dense)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if strided:
        if t.numel() and (any(st < 0 for st in t.stride())
                          or (t.dim() == 3 and t.stride(2) != 1 and t.shape[2] > 1)):
            raise ValueError(f"{name} must have non-negative strides and contiguous channels")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (dense row-major)")
    return t.data_ptr()


def _flat(t, name, shape):
    """t seen with `shape` without a copy: the library keeps only the data
    pointer, and a temporary copy would go back to torch's allocator before
    the queued kernel reads it."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (its data is read in place)")
    if t.numel() != math.prod(shape):
        raise ValueError(f"{name} has {t.numel()} elements, expected {math.prod(shape)}")
    return t.view(shape)


def kda_chunk_prefill_fwd(q, k, v, g, beta_logits, A_log, dt_bias, lower_bound: float,
                          scale: float, initial_state, cu_seqlens, out, final_state, workspace,
                          stream=None, checkpoints=None, checkpoint_interval: int = 0) -> None:
    """Queue one KDA chunked-prefill forward (see include/kda.h for the contract).

    q, k, v, g, out [T, H, 128] bf16; beta_logits [T, H] bf16; A_log [H] fp32;
    dt_bias [H, 128] fp32; initial_state None or [N, H, 128, 128]; final_state
    [N, H, 128, 128] (fp32 or bf16, the same dtype as initial_state);
    cu_seqlens [N + 1] int32; workspace uint8 (or None if no workspace is
    needed); stream: a torch.cuda.Stream, a raw hipStream_t int, or None for
    torch's current stream.  Leading singleton batch dims ([1, T, H, 128]) are
    accepted.  checkpoints: None, or [C, H, 128, 128] in the state dtype to
    receive the state after every checkpoint_interval tokens of each sequence
    (kda_chunk_prefill_fwd_checkpoints; C >= T // checkpoint_interval).
    """
    import torch
    lib = load_library()

    def squeeze_batch(t):
        return t[0] if (t is not None and t.dim() == 4 and t.shape[0] == 1
                        and t.shape[-1] == HEAD_DIM and t.shape[-2] != HEAD_DIM) else t

    q, k, v, g, out = (squeeze_batch(t) for t in (q, k, v, g, out))
    if q.dim() != 3:
        raise ValueError(f"q must be [T, H, {HEAD_DIM}], got {tuple(q.shape)}")
    T, H, D = q.shape
    if D != HEAD_DIM:
        raise ValueError(f"head_dim must be {HEAD_DIM}, got {D}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [N + 1] with N >= 1")
    N = cu_seqlens.numel() - 1
    bf = torch.bfloat16
    if final_state.dtype == torch.float32:
        sdt = KDA_STATE_FP32
    elif final_state.dtype == torch.bfloat16:
        sdt = KDA_STATE_BF16
    else:
        raise TypeError(f"state dtype must be float32 or bfloat16, got {final_state.dtype}")
    sshape = (N, H, HEAD_DIM, HEAD_DIM)
    if beta_logits.dim() == 3 and beta_logits.shape[0] == 1:
        beta_logits = beta_logits[0]
    if beta_logits.dim() == 3 and beta_logits.shape[-1] == 1:
        beta_logits = beta_logits[..., 0]
    views = {"q": q, "k": k, "v": v, "g": g, "beta": beta_logits, "out": out}
    ptrs = [
        _check(q, "q", bf, (T, H, D), strided=True), _check(k, "k", bf, (T, H, D), strided=True),
        _check(v, "v", bf, (T, H, D), strided=True), _check(g, "g", bf, (T, H, D), strided=True),
        _check(beta_logits, "beta_logits", bf, (T, H), strided=True),
        _check(_flat(A_log, "A_log", (H,)), "A_log", torch.float32, (H,)),
        _check(_flat(dt_bias, "dt_bias", (H, D)), "dt_bias", torch.float32, (H, D)),
    ]
    s0 = None if initial_state is None else _check(initial_state, "initial_state",
                                                   final_state.dtype, sshape)
    cu = _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    o = _check(out, "out", bf, (T, H, D), strided=True)
    fs = _check(final_state, "final_state", final_state.dtype, sshape)
    if workspace is None:
        ws, wsb = None, 0
    else:
        ws = _check(workspace, "workspace", torch.uint8)
        wsb = workspace.numel()
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    args = (*ptrs, float(lower_bound), float(scale), s0, cu, o, fs, ws,
            ctypes.c_void_p(int(stream)), T, H, N, sdt, wsb)
    st = None
    if not all(t.is_contiguous() for t in views.values()):
        st = _Strides()
        for name in ("q", "k", "v", "g", "out"):
            setattr(st, f"{name}_token", views[name].stride(0))
            setattr(st, f"{name}_head", views[name].stride(1))
        st.beta_token, st.beta_head = views["beta"].stride(0), views["beta"].stride(1)
    if checkpoints is not None:
        if checkpoints.dim() != 4:
            raise ValueError("checkpoints must be [C, H, 128, 128]")
        ck = _check(checkpoints, "checkpoints", final_state.dtype,
                    (checkpoints.shape[0], H, HEAD_DIM, HEAD_DIM))
        rc = lib.kda_chunk_prefill_fwd_checkpoints(
            *args, None if st is None else ctypes.byref(st), ck, int(checkpoint_interval),
            int(checkpoints.shape[0]))
    elif st is None:
        rc = lib.kda_chunk_prefill_fwd(*args)
    else:
        rc = lib.kda_chunk_prefill_fwd_strided(*args, ctypes.byref(st))
    if rc != KDA_OK:
        detail = lib.kda_last_hip_error().decode() if rc == 4 else ""
        raise KdaError(rc, f"kda_chunk_prefill_fwd: {kda_status_string(rc)} {detail}".strip())


def kda_spec_decode_step(q, k, v, g, beta_logits, A_log, dt_bias, lower_bound: float, scale: float,
                         state_pool, cu_seqlens, state_indices, num_accepted_tokens, out, workspace,
                         stream=None) -> None:
    """Queue one speculative-decode step with num_accepted_tokens rollback (see
    include/kda.h, kda_spec_decode_step).

    q, k, v, g, out [T, H, 128] bf16 (dense); beta_logits [T, H] bf16;
    state_pool [num_slots, H, 128, 128] fp32 or bf16 (read and written in
    place); cu_seqlens [N + 1] int32; state_indices [N, S] int32;
    num_accepted_tokens [N] int32; workspace uint8.
    """
    import torch
    lib = load_library()
    if q.dim() != 3:
        raise ValueError(f"q must be [T, H, {HEAD_DIM}], got {tuple(q.shape)}")
    T, H, D = q.shape
    if D != HEAD_DIM:
        raise ValueError(f"head_dim must be {HEAD_DIM}, got {D}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [N + 1] with N >= 1")
    N = cu_seqlens.numel() - 1
    bf = torch.bfloat16
    if state_pool.dtype == torch.float32:
        sdt = KDA_STATE_FP32
    elif state_pool.dtype == torch.bfloat16:
        sdt = KDA_STATE_BF16
    else:
        raise TypeError(f"state dtype must be float32 or bfloat16, got {state_pool.dtype}")
    if state_pool.dim() != 4:
        raise ValueError("state_pool must be [num_slots, H, 128, 128]")
    if state_indices.dim() != 2 or state_indices.shape[0] != N:
        raise ValueError(f"state_indices must be [N, S] with N = {N}")
    ptrs = [_check(t, n, bf, (T, H, D)) for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"))]
    ptrs += [_check(beta_logits, "beta_logits", bf, (T, H)),
             _check(_flat(A_log, "A_log", (H,)), "A_log", torch.float32, (H,)),
             _check(_flat(dt_bias, "dt_bias", (H, D)), "dt_bias", torch.float32, (H, D))]
    pool = _check(state_pool, "state_pool", state_pool.dtype,
                  (state_pool.shape[0], H, HEAD_DIM, HEAD_DIM))
    cu = _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    idx = _check(state_indices, "state_indices", torch.int32, tuple(state_indices.shape))
    acc = _check(num_accepted_tokens, "num_accepted_tokens", torch.int32, (N,))
    o = _check(out, "out", bf, (T, H, D))
    ws = _check(workspace, "workspace", torch.uint8)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    rc = lib.kda_spec_decode_step(*ptrs, float(lower_bound), float(scale), pool,
                                  int(state_pool.shape[0]), cu, idx, int(state_indices.shape[1]),
                                  acc, o, ws, ctypes.c_void_p(int(stream)), T, H, N, sdt,
                                  workspace.numel())
    if rc != KDA_OK:
        detail = lib.kda_last_hip_error().decode() if rc == 4 else ""
        raise KdaError(rc, f"kda_spec_decode_step: {kda_status_string(rc)} {detail}".strip())


def kda_chunk_prefill_fwd_noalloc(q, k, v, g, beta_logits, A_log, dt_bias, lower_bound: float,
                                  scale: float, initial_state, cu_seqlens, out, final_state, status,
                                  stream=None) -> None:
    """kda_chunk_prefill_fwd without a workspace (see include/kda.h,
    kda_chunk_prefill_fwd_noalloc): dense tensors as for the forward call;
    status a device int32 tensor of one element (the status word)."""
    import torch
    lib = load_library()
    if q.dim() != 3:
        raise ValueError(f"q must be [T, H, {HEAD_DIM}], got {tuple(q.shape)}")
    T, H, D = q.shape
    if D != HEAD_DIM:
        raise ValueError(f"head_dim must be {HEAD_DIM}, got {D}")
    N = cu_seqlens.numel() - 1
    if N < 1:
        raise ValueError("cu_seqlens must be [N + 1] with N >= 1")
    bf = torch.bfloat16
    if final_state.dtype == torch.float32:
        sdt = KDA_STATE_FP32
    elif final_state.dtype == torch.bfloat16:
        sdt = KDA_STATE_BF16
    else:
        raise TypeError(f"state dtype must be float32 or bfloat16, got {final_state.dtype}")
    sshape = (N, H, HEAD_DIM, HEAD_DIM)
    ptrs = [_check(t, n, bf, (T, H, D)) for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"))]
    ptrs += [_check(beta_logits, "beta_logits", bf, (T, H)),
             _check(_flat(A_log, "A_log", (H,)), "A_log", torch.float32, (H,)),
             _check(_flat(dt_bias, "dt_bias", (H, D)), "dt_bias", torch.float32, (H, D))]
    s0 = None if initial_state is None else _check(initial_state, "initial_state",
                                                   final_state.dtype, sshape)
    cu = _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    o = _check(out, "out", bf, (T, H, D))
    fs = _check(final_state, "final_state", final_state.dtype, sshape)
    st = _check(status, "status", torch.int32, (1,))
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    rc = lib.kda_chunk_prefill_fwd_noalloc(*ptrs, float(lower_bound), float(scale), s0, cu, o, fs, st,
                                           ctypes.c_void_p(int(stream)), T, H, N, sdt)
    if rc != KDA_OK:
        detail = lib.kda_last_hip_error().decode() if rc == 4 else ""
        raise KdaError(rc, f"kda_chunk_prefill_fwd_noalloc: {kda_status_string(rc)} {detail}".strip())


def kda_gate_proj_workspace_size(num_tokens: int, hidden_dim: int, n_ab: int) -> int:
    return int(load_library().kda_gate_proj_workspace_size(int(num_tokens), int(hidden_dim),
                                                             int(n_ab)))


def kda_gate_proj(hidden, w_ab, w_b, p_ab, g, workspace, stream=None) -> None:
    """Queue the gate / beta projections (see include/kda.h, kda_gate_proj):
    P = bf16(hidden w_ab^T) into p_ab [M, n_ab], G = bf16(P[:, :128] w_b^T)
    into g [M, n_b] (or a [M, n_b / 128, 128] view).  bf16 tensors, dense;
    workspace uint8 of kda_gate_proj_workspace_size bytes (no initialisation
    needed)."""
    import torch
    lib = load_library()
    bf = torch.bfloat16
    if hidden.dim() != 2 or w_ab.dim() != 2 or w_b.dim() != 2:
        raise ValueError("hidden, w_ab and w_b must be 2-D")
    M, K = hidden.shape
    n_ab, n_b = w_ab.shape[0], w_b.shape[0]
    ptrs = [_check(hidden, "hidden", bf, (M, K)), _check(w_ab, "w_ab", bf, (n_ab, K)),
            _check(w_b, "w_b", bf, (n_b, 128)), _check(p_ab, "p_ab", bf, (M, n_ab)),
            _check(g.reshape(M, n_b) if g.is_contiguous() else g, "g", bf, (M, n_b))]
    ws = _check(workspace, "workspace", torch.uint8)
    if stream is None:
        stream = torch.cuda.current_stream(hidden.device).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    rc = lib.kda_gate_proj(*ptrs, ws, workspace.numel(), ctypes.c_void_p(int(stream)), M, K, n_ab,
                           n_b)
    if rc != KDA_OK:
        detail = lib.kda_last_hip_error().decode() if rc == 4 else ""
        raise KdaError(rc, f"kda_gate_proj: {kda_status_string(rc)} {detail}".strip())


# ---- include/kda_layer.h: the operators around the forward --------------------
#
# Their calls take microseconds on the device, so the checks are kept short: a
# tensor is compared as a whole in the path that passes, and what is wrong with
# it is found out in _refuse.

def _torch():
    """torch, imported on first use (like load_library)."""
    global _torch_module, _raw_stream, _device
    if _torch_module is None:
        import torch
        _raw_stream, _device = _queries(torch)
        _torch_module = torch
    return _torch_module


def _queries(torch):
    """(handle of the current stream of GPU i, index of the current GPU) as
    functions: torch's own short forms of the public calls, 1.2 us less per call,
    and the public ones in a torch that does not have them."""
    c, cuda = torch._C, torch.cuda
    return (getattr(c, "_cuda_getCurrentRawStream", None) or (lambda i: cuda.current_stream(i).cuda_stream),
            getattr(c, "_cuda_getDevice", None) or cuda.current_device)


_torch_module = _raw_stream = _device = None


def _refuse(t, name, dtype, shape, index):
    """Raise what is wrong with t (see _on)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    raise ValueError(f"{name} must be contiguous (dense row-major)")


def _view(t, name, dtype, shape, index):
    """Device pointer of t, whose strides are the caller's to look at."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index:
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, index)


def _on(t, name, dtype, shape, index):
    """Device pointer of t: dense, of this dtype and shape, on GPU `index`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, index)


def _gpu(t, name):
    """Index of the GPU t is on."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    return t.get_device()


def _call(name, fn, index, stream, before, after):
    """fn(*before, stream, *after) on GPU `index`; raises on a refusal."""
    if stream is None:
        stream = _raw_stream(index)
    elif isinstance(stream, _torch_module.cuda.Stream):
        stream = stream.cuda_stream
    if index == _device():
        rc = fn(*before, stream, *after)
    else:
        with _torch_module.cuda.device(index):
            rc = fn(*before, stream, *after)
    if rc != KDA_OK:
        detail = kda_last_hip_error() if rc == 4 else ""
        raise KdaError(rc, f"{name}: {kda_status_string(rc)} {detail}".strip())


def _state_dtype(t):
    torch = _torch()
    dtype = t.dtype if isinstance(t, torch.Tensor) else type(t)
    if dtype == torch.float32:
        return KDA_STATE_FP32
    if dtype == torch.bfloat16:
        return KDA_STATE_BF16
    raise TypeError(f"state dtype must be float32 or bfloat16, got {dtype}")


@functools.lru_cache(maxsize=256)
def _gdr_strides(one_row, one_key_head, one_value_head, q, k, v, a, beta_logits, out):
    """kda_gdr_strides_t of tensors with these strides (0 for a dimension of one
    element, whose stride means nothing); None where channels are not adjacent."""
    if any(st[2] != 1 for st in (q, k, v, out)):
        return None
    flat = []
    for st, one_head in ((q, one_key_head), (k, one_key_head), (v, one_value_head),
                         (a, one_value_head), (beta_logits, one_value_head), (out, one_value_head)):
        flat += [0 if one_row else st[0], 0 if one_head else st[1]]
    return _GdrStrides(*flat)


def _gdr_rows(q, k, v, a, beta_logits, A_log, dt_bias, out):
    """(pointers of the inputs, pointer of out, GPU, rows, key heads, value heads, strides)."""
    dev = _gpu(q, "q")
    torch = _torch_module
    bf, f32 = torch.bfloat16, torch.float32
    if q.dim() != 3 or q.shape[2] != HEAD_DIM:
        raise ValueError(f"q must be [T, Hk, {HEAD_DIM}], got {tuple(q.shape)}")
    if not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError(f"v must be [T, Hv, {HEAD_DIM}]")
    T, hk, _ = rows = q.shape
    hv = v.shape[1]
    heads, gates, per_head = (T, hv, HEAD_DIM), (T, hv), (hv,)
    ptrs = (_view(q, "q", bf, rows, dev), _view(k, "k", bf, rows, dev), _view(v, "v", bf, heads, dev),
            _view(a, "a", bf, gates, dev), _view(beta_logits, "beta_logits", bf, gates, dev),
            _on(A_log, "A_log", f32, per_head, dev), _on(dt_bias, "dt_bias", f32, per_head, dev))
    o = _view(out, "out", bf, heads, dev)
    st = _gdr_strides(T <= 1, hk == 1, hv == 1, q.stride(), k.stride(), v.stride(), a.stride(),
                      beta_logits.stride(), out.stride())
    if st is None:
        raise ValueError("q, k, v and out must have contiguous channels")
    return ptrs, o, dev, T, hk, hv, st


def kda_gdr_get_workspace_size(max_tokens: int, key_heads: int, value_heads: int,
                               max_seqs: int) -> int:
    return int(load_library().kda_gdr_get_workspace_size(int(max_tokens), int(key_heads),
                                                         int(value_heads), int(max_seqs)))


def kda_gdr_prefill_fwd(q, k, v, a, beta_logits, A_log, dt_bias, scale: float, initial_state,
                        cu_seqlens, out, final_state, workspace, stream=None) -> None:
    """Queue one prefill of the gated delta rule with one decay per value head
    (see include/kda_layer.h, kda_gdr_prefill_fwd).

    q, k [T, Hk, 128], v, out [T, Hv, 128] bf16 and a, beta_logits [T, Hv] bf16,
    strided views among them (channels contiguous, strides multiples of 8);
    A_log, dt_bias [Hv] fp32; initial_state None or [N, Hv, 128, 128];
    final_state [N, Hv, 128, 128] fp32 or bf16, initial_state's dtype (and may
    be it); cu_seqlens [N + 1] int32; workspace uint8 of
    kda_gdr_get_workspace_size(T, Hk, Hv, N) bytes, no initialisation needed;
    stream as for kda_chunk_prefill_fwd.
    """
    lib = load_library()
    ptrs, o, dev, T, hk, hv, st = _gdr_rows(q, k, v, a, beta_logits, A_log, dt_bias, out)
    torch = _torch_module
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [N + 1] with N >= 1")
    n = cu_seqlens.numel() - 1
    shape = (n, hv, HEAD_DIM, HEAD_DIM)
    sdt = _state_dtype(final_state)
    s0 = None if initial_state is None else _on(initial_state, "initial_state", final_state.dtype,
                                                shape, dev)
    cu = _on(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), dev)
    fs = _on(final_state, "final_state", final_state.dtype, shape, dev)
    ws, size = None, 0
    if workspace is not None:
        size = workspace.numel()
        ws = _on(workspace, "workspace", torch.uint8, (size,), dev)
    _call("kda_gdr_prefill_fwd", lib.kda_gdr_prefill_fwd, dev, stream,
          (*ptrs, scale, s0, cu, o, fs, ws), (T, hk, hv, n, sdt, size, st))


def kda_gdr_decode_step(q, k, v, a, beta_logits, A_log, dt_bias, scale: float, state_pool,
                        state_indices, out, stream=None) -> None:
    """Queue one token of the gated delta rule for each of N sequences on a
    pool of states, in place (see include/kda_layer.h, kda_gdr_decode_step).

    q, k, v, a, beta_logits, out as for kda_gdr_prefill_fwd with T = N;
    state_pool [num_slots, Hv, 128, 128] fp32 or bf16; state_indices [N] int32,
    an index outside the pool marks a padding row.
    """
    lib = load_library()
    ptrs, o, dev, n, hk, hv, st = _gdr_rows(q, k, v, a, beta_logits, A_log, dt_bias, out)
    sdt = _state_dtype(state_pool)
    if state_pool.dim() != 4:
        raise ValueError("state_pool must be [num_slots, Hv, 128, 128]")
    slots = state_pool.shape[0]
    pool = _on(state_pool, "state_pool", state_pool.dtype, (slots, hv, HEAD_DIM, HEAD_DIM), dev)
    idx = _on(state_indices, "state_indices", _torch_module.int32, (n,), dev)
    _call("kda_gdr_decode_step", lib.kda_gdr_decode_step, dev, stream,
          (*ptrs, scale, pool, slots, idx, o), (n, hk, hv, sdt, st))


def _row_stride(t, name):
    """Elements between the rows of a 2-D tensor whose rows are dense."""
    if t.is_contiguous():
        return t.shape[1]
    row, col = t.stride()
    if col != 1 and t.shape[1] > 1 and t.shape[0]:
        raise ValueError(f"{name} must have contiguous rows")
    return row


def kda_add_rms_norm(x, residual, weight, eps: float, out, out_scale=None, group_size: int = 0,
                     stream=None) -> None:
    """Queue residual <- x + residual and out <- its RMS norm (see
    include/kda_layer.h, kda_add_rms_norm).

    x, residual (or None) [M, dim] bf16, rows may be strided; weight [dim]
    bf16; out [M, dim] bf16, or float8_e4m3fn with out_scale fp32 [M, 1] (or
    [M]; group_size 0) or [M, ceil(dim / 128)] (group_size 128).
    """
    lib = load_library()
    dev = _gpu(x, "x")
    torch = _torch_module
    bf = torch.bfloat16
    if x.dim() != 2:
        raise ValueError(f"x must be [M, dim], got {tuple(x.shape)}")
    shape = x.shape
    m, dim = shape
    fp8 = isinstance(out, torch.Tensor) and out.dtype == torch.float8_e4m3fn
    xp = _view(x, "x", bf, shape, dev)
    op = _view(out, "out", torch.float8_e4m3fn if fp8 else bf, shape, dev)
    rp = rs = 0
    if residual is not None:
        rp = _view(residual, "residual", bf, shape, dev)
        rs = _row_stride(residual, "residual")
    w = _on(weight, "weight", bf, (dim,), dev)
    sc = None
    if out_scale is not None:
        groups = (dim + 127) // 128 if group_size else 1
        flat = groups == 1 and isinstance(out_scale, torch.Tensor) and out_scale.dim() == 1
        sc = _on(out_scale, "out_scale", torch.float32, (m,) if flat else (m, groups), dev)
    _call("kda_add_rms_norm", lib.kda_add_rms_norm, dev, stream, (xp, rp, w, eps, op, sc),
          (m, dim, _row_stride(x, "x"), rs, _row_stride(out, "out"), 1 if fp8 else 0, group_size))


def kda_w4_proj(x, w, scales, zeros, y, group_size: int, stream=None) -> None:
    """Queue y = x (4-bit weights)^T for at most 64 tokens (see
    include/kda_layer.h, kda_w4_proj).

    x [M, K] and y [M, N] bf16, rows may be strided; w [N, K / 2] uint8, even k
    in the low four bits; scales [N, K / group_size] bf16; zeros the same or
    None (8 everywhere).
    """
    lib = load_library()
    dev = _gpu(x, "x")
    torch = _torch_module
    bf = torch.bfloat16
    if x.dim() != 2 or not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("x and w must be 2-D tensors")
    m, k = x.shape
    n = w.shape[0]
    if group_size not in (32, 64, 128) or k % group_size:
        raise ValueError(f"group_size must be 32, 64 or 128 and divide {k}, got {group_size}")
    per = (n, k // group_size)
    ptrs = (_view(x, "x", bf, (m, k), dev), _on(w, "w", torch.uint8, (n, k // 2), dev),
            _on(scales, "scales", bf, per, dev),
            None if zeros is None else _on(zeros, "zeros", bf, per, dev),
            _view(y, "y", bf, (m, n), dev))
    _call("kda_w4_proj", lib.kda_w4_proj, dev, stream, ptrs,
          (m, k, n, group_size, _row_stride(x, "x"), _row_stride(y, "y")))


# ---- include/kda_mx4.h: microscaled 4-bit numbers ------------------------------

def _columns(k, name):
    if k % 32 or k <= 0:
        raise ValueError(f"{name} must have a multiple of 32 columns, got {k}")


def kda_mx4_quant(x, codes, scales, stream=None) -> None:
    """Queue codes, scales <- x as microscaled 4-bit numbers (see
    include/kda_mx4.h, kda_mx4_quant).

    x [M, k] bf16, rows may be strided (by multiples of 8); codes [M, k / 2] and
    scales [M, k / 32] uint8, dense.
    """
    lib = load_library()
    dev = _gpu(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be [M, k], got {tuple(x.shape)}")
    m, k = shape = x.shape
    _columns(k, "x")
    u8 = _torch_module.uint8
    ptrs = (_view(x, "x", _torch_module.bfloat16, shape, dev), _on(codes, "codes", u8, (m, k // 2), dev),
            _on(scales, "scales", u8, (m, k // 32), dev))
    _call("kda_mx4_quant", lib.kda_mx4_quant, dev, stream, ptrs, (m, k, _row_stride(x, "x")))


def kda_mx4_dequant(codes, scales, out, stream=None) -> None:
    """Queue out <- the values of codes and scales (see include/kda_mx4.h,
    kda_mx4_dequant).  Shapes as for kda_mx4_quant, out [M, k] bf16."""
    lib = load_library()
    dev = _gpu(out, "out")
    if out.dim() != 2:
        raise ValueError(f"out must be [M, k], got {tuple(out.shape)}")
    m, k = shape = out.shape
    _columns(k, "out")
    u8 = _torch_module.uint8
    ptrs = (_on(codes, "codes", u8, (m, k // 2), dev), _on(scales, "scales", u8, (m, k // 32), dev),
            _view(out, "out", _torch_module.bfloat16, shape, dev))
    _call("kda_mx4_dequant", lib.kda_mx4_dequant, dev, stream, ptrs, (m, k, _row_stride(out, "out")))


def kda_mx4_proj(x, x_scales, w, w_scales, y, stream=None) -> None:
    """Queue y = x w^T with microscaled 4-bit weights (see include/kda_mx4.h,
    kda_mx4_proj).

    x [M, k] bf16 with x_scales None (M <= 64, rows may be strided), or codes
    [M, k / 2] with x_scales [M, k / 32]; w [n, k / 2] and w_scales [n, k / 32]
    uint8; y [M, n] bf16, rows may be strided.
    """
    lib = load_library()
    dev = _gpu(x, "x")
    torch = _torch_module
    if x.dim() != 2 or not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("x and w must be 2-D tensors")
    m, k = x.shape
    n, u8 = w.shape[0], torch.uint8
    if x_scales is None:
        _columns(k, "x")
        xp, xs, row = _view(x, "x", torch.bfloat16, (m, k), dev), None, _row_stride(x, "x")
    else:
        k *= 2
        _columns(k, "x (of values)")
        xp, xs, row = _on(x, "x", u8, (m, k // 2), dev), _on(x_scales, "x_scales", u8, (m, k // 32), dev), 0
    ptrs = (xp, xs, _on(w, "w", u8, (n, k // 2), dev), _on(w_scales, "w_scales", u8, (n, k // 32), dev),
            _view(y, "y", torch.bfloat16, (m, n), dev))
    _call("kda_mx4_proj", lib.kda_mx4_proj, dev, stream, ptrs, (m, k, n, row, _row_stride(y, "y")))


def kda_mx4_moe_workspace_size(max_tokens: int, k: int, inter: int, experts: int, shared: int,
                               top_k: int) -> int:
    return int(load_library().kda_mx4_moe_workspace_size(int(max_tokens), int(k), int(inter), int(experts),
                                                         int(shared), int(top_k)))


_SCORING = {"sigmoid": 0, "softmax": 1}


def kda_mx4_moe(x, router, router_bias, w_up, w_up_scales, w_down, w_down_scales, out, expert_ids,
                expert_gates, workspace, scoring: str = "sigmoid", renormalise: bool = True,
                route_scale: float = 1.0, state_indices=None, stream=None) -> None:
    """Queue a mixture-of-experts layer for at most 64 tokens (see
    include/kda_mx4.h, kda_mx4_moe).

    x, out [M, k] bf16, rows may be strided (by multiples of 8); router [E, k]
    bf16; router_bias [E] fp32 or None; w_up [E + S, 2 inter, k / 2], w_down
    [E + S, k, inter / 2] uint8 with their scales ([..., k / 32], [..., inter /
    32]), the last S experts shared by every token; expert_ids int32 and
    expert_gates fp32 [M, top_k], written; workspace uint8 of
    kda_mx4_moe_workspace_size(M, k, inter, E, S, top_k) bytes, no initialisation
    needed; state_indices None or [M] int32, an index below zero marks a padding
    row.
    """
    lib = load_library()
    dev = _gpu(x, "x")
    torch = _torch_module
    bf = torch.bfloat16
    for t, name, dims in ((x, "x", 2), (router, "router", 2), (w_up, "w_up", 3), (expert_ids, "expert_ids", 2)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name} must be a tensor of {dims} dimensions")
    m, k = rows = x.shape
    experts, (every, twice, _), top = router.shape[0], w_up.shape, expert_ids.shape[1]
    inter, shared = twice // 2, every - experts
    _columns(k, "x")
    if twice % 64 or shared < 0:
        raise ValueError(f"w_up must be [E + S, 2 inter, k / 2] with E = {experts} and inter a multiple of 32, "
                         f"got {tuple(w_up.shape)}")
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be sigmoid or softmax, got {scoring!r}")
    size = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
    u8 = torch.uint8
    ptrs = (_view(x, "x", bf, rows, dev), _on(router, "router", bf, (experts, k), dev),
            None if router_bias is None else _on(router_bias, "router_bias", torch.float32, (experts,), dev),
            _on(w_up, "w_up", u8, (every, twice, k // 2), dev),
            _on(w_up_scales, "w_up_scales", u8, (every, twice, k // 32), dev),
            _on(w_down, "w_down", u8, (every, k, inter // 2), dev),
            _on(w_down_scales, "w_down_scales", u8, (every, k, inter // 32), dev),
            None if state_indices is None else _on(state_indices, "state_indices", torch.int32, (m,), dev),
            _view(out, "out", bf, rows, dev), _on(expert_ids, "expert_ids", torch.int32, (m, top), dev),
            _on(expert_gates, "expert_gates", torch.float32, (m, top), dev),
            _on(workspace, "workspace", u8, (size,), dev))
    _call("kda_mx4_moe", lib.kda_mx4_moe, dev, stream, ptrs,
          (m, k, inter, experts, shared, top, _row_stride(x, "x"), _row_stride(out, "out"), _SCORING[scoring],
           1 if renormalise else 0, route_scale, size))
