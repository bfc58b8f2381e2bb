"""Thin Python binding of libkda (include/kda.h), same names as the C ABI.

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, outputs are allocated with torch when the caller passes none, and
the raw device pointers go to the C entry points on the current CUDA stream.
Every step of the computation runs inside libkda's kernels.  If the shared
library is missing the import of this module's functions fails loudly; there
is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_BF16, KDA_F32 = 0, 1
KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_MISALIGNED = 0, 1, 2, 3
KDA_ERR_CUDA, KDA_ERR_TIMEOUT, KDA_ERR_WORKSPACE, KDA_STATUS_GATE_RANGE = 4, 5, 6, 7
KDA_STATUS_SLOT_RANGE, KDA_ERR_SCRATCH_TOO_SMALL, KDA_STATUS_POSITION_RANGE = 8, 9, 10
KDA_NOALLOC_SCRATCH_BYTES = 128 << 20
KDA_OP_CHUNK, KDA_OP_VARLEN, KDA_OP_DECODE, KDA_OP_BWD, KDA_OP_CHUNK_BWD = 0, 1, 2, 3, 4
KDA_GATE_CHANNEL, KDA_GATE_HEAD, KDA_GATE_NONE = 0, 1, 2
KDA_ACT_NONE, KDA_ACT_SILU = 0, 1
KDA_NORM_NONE, KDA_NORM_RMS, KDA_NORM_L2 = 0, 1, 2
KDA_ROT_HALF, KDA_ROT_PAIRS = 0, 1

_lib = None


class KdaError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {kda_status_string(code)} (code {code})")
        self.code = code


def lib() -> ctypes.CDLL:
    """The loaded libkda.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libkda.so not found at {LIB_PATH}; build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.kda_chunk_fwd.argtypes = [P, P, P, P, P, P, P, P, I, I64, I, I, I, I, I, I, P, SZ, P]
        L.kda_varlen_fwd.argtypes = [P, P, P, P, P, P, I, I64, I, I, I, I, P, P, I64, P, P, P, I, I, P, SZ, P]
        L.kda_decode_step.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P]
        L.kda_decode_step_bf16state.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P]
        L.kda_gdn_chunk_fwd.argtypes = L.kda_chunk_fwd.argtypes
        L.kda_gdn_varlen_fwd.argtypes = L.kda_varlen_fwd.argtypes
        L.kda_gdn_decode_step.argtypes = L.kda_decode_step.argtypes
        L.kda_gdn_decode_step_bf16state.argtypes = L.kda_decode_step.argtypes
        L.kda_chunk_fwd_host.argtypes = [P, P, P, P, P, P, P, P, I, I64, I, I, I, I, I, I64, P, SZ, P]
        L.kda_host_fwd_workspace_size.argtypes = [I, I, I, I, I64, I, I]
        L.kda_host_fwd_workspace_size.restype = SZ
        L.kda_bwd.argtypes = [P, P, P, P, I, P, P, P, P, P, I, I64, I, I, I, P, P, P, P, P, P, I, P, SZ, P]
        L.kda_bwd_noalloc.argtypes = [P, P, P, P, I, P, P, P, P, P, I, I64, I, I, I, P, P, P, P, P, P, I, P]
        L.kda_chunk_bwd.argtypes = [P, P, P, P, I, P, P, P, P, P, I, I64, I, I, I, I, P, P, P, P, P, P, I, P, SZ,
                                    P]
        L.kda_varlen_fwd_pool.argtypes = [P, P, P, P, I, P, P, I, I64, I, I, I, I, P, I64, I, P, I64, P, P, P, P, I,
                                          I, P, SZ, P]
        L.kda_snapshot_count.argtypes = [I64, I64]
        L.kda_snapshot_count.restype = I64
        L.kda_snapshot_offsets.argtypes = [P, I, I64, P]
        L.kda_snapshot_lookup.argtypes = [P, I, I, I64, I64, P]
        L.kda_snapshot_lookup.restype = I64
        L.kda_workspace_size.argtypes = [I, I, I64, I, I, I, I]
        L.kda_workspace_size.restype = SZ
        L.kda_status_string.argtypes = [I]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_get_device_status.argtypes = [P]
        L.kda_selftest_bounded_wait.argtypes = [P]
        F = ctypes.c_float
        L.kda_conv_fwd.argtypes = [P, I64, P, P, P, P, P, P, I, I64, I, I, I, I, I, P]
        L.kda_conv_step.argtypes = [P, I64, P, P, P, P, I, I, I, I, I, I, P]
        L.kda_conv_bwd.argtypes = [P, I64, P, P, P, P, P, P, I, I64, I, I, I, P, P, P, P, I, I, P, SZ, P]
        L.kda_conv_bwd_workspace_size.argtypes = [I64, I, I]
        ssm_in = [P, I64, P, I64, P, P, I64, P, I64, P, P, I64, P, I]  # u .. delta_softplus
        L.kda_ssm_fwd.argtypes = ssm_in + [P, P, P, P, I, I64, I, I, I, I, I, P, SZ, P]
        L.kda_ssm_step.argtypes = ssm_in + [P, P, I, I, I, I, I, I, P]
        L.kda_ssm_bwd.argtypes = ssm_in + [P, P, P, P, I, I64, I, I, I, P, P, P, P, P, P, P, P, P, I, I, P, SZ, P]
        L.kda_ssm_fwd_workspace_size.argtypes = L.kda_ssm_bwd_workspace_size.argtypes = [I, I64, I, I, I, I]
        L.kda_qk_norm_fwd.argtypes = [P, I64, P, I64, P, P, P, P, P, I64, P, P, I64, I, I, I, I, I, I, F, I, I, P]
        L.kda_qk_norm_bwd.argtypes = [P, I64, P, I64, P, P, P, P, P, P, P, I64, P, P, P, P, I64, I, I, I, I, I, I, F,
                                      I, I, P, SZ, P]
        L.kda_qk_norm_bwd_workspace_size.argtypes = [I]
        for f in (L.kda_conv_bwd_workspace_size, L.kda_ssm_fwd_workspace_size, L.kda_ssm_bwd_workspace_size,
                  L.kda_qk_norm_bwd_workspace_size):
            f.restype = SZ
        for f in (L.kda_conv_fwd, L.kda_conv_step, L.kda_conv_bwd, L.kda_ssm_fwd, L.kda_ssm_step, L.kda_ssm_bwd,
                  L.kda_qk_norm_fwd, L.kda_qk_norm_bwd):
            f.restype = I
        for f in (L.kda_chunk_fwd, L.kda_varlen_fwd, L.kda_decode_step, L.kda_decode_step_bf16state,
                  L.kda_gdn_chunk_fwd, L.kda_gdn_varlen_fwd, L.kda_gdn_decode_step, L.kda_varlen_fwd_pool, L.kda_bwd,
                  L.kda_bwd_noalloc, L.kda_chunk_bwd, L.kda_selftest_bounded_wait, L.kda_gdn_decode_step_bf16state,
                  L.kda_chunk_fwd_host,
                  L.kda_snapshot_offsets,
                  L.kda_get_device_status):
            f.restype = I
        _lib = L
    return _lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use bfloat16 or float32")


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libkda must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _same_device(dev: int, what: str) -> None:
    """The library launches on the current device: the tensors, and with them the stream, must be that one's."""
    if dev != torch.cuda.current_device():
        raise ValueError(f"{what} cuda:{dev}, but the current device is cuda:{torch.cuda.current_device()}: "
                         "call under torch.cuda.device")


def _stream(device) -> ctypes.c_void_p:
    if device is not None and device.index is not None:
        _same_device(device.index, "the tensors are on")
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(rc: int, where: str):
    if rc != KDA_OK:
        raise KdaError(rc, where)


def _dtype_of(code: int):
    return torch.bfloat16 if code == KDA_BF16 else torch.float32


def kda_status_string(code: int) -> str:
    return lib().kda_status_string(int(code)).decode()


def kda_snapshot_count(seqlen: int, interval: int) -> int:
    return int(lib().kda_snapshot_count(int(seqlen), int(interval)))


def kda_snapshot_offsets(cu_seqlens_host, interval: int) -> torch.Tensor:
    """HOST int64 [N+1] snapshot offsets for HOST cu_seqlens (a list or CPU tensor)."""
    cu = torch.as_tensor(cu_seqlens_host, dtype=torch.int64).cpu().contiguous()
    N = cu.numel() - 1
    off = torch.empty(N + 1, dtype=torch.int64)
    _check(lib().kda_snapshot_offsets(_ptr(cu), N, int(interval), _ptr(off)), "kda_snapshot_offsets")
    return off


def kda_snapshot_lookup(offsets_host, seq: int, interval: int, prefix_len: int):
    """(index, covered): the latest snapshot of sequence `seq` covering at most `prefix_len`
    tokens (index into the packed snapshots, tokens it covers), or (-1, 0) if there is none."""
    off = torch.as_tensor(offsets_host, dtype=torch.int64).cpu().contiguous()
    cov = ctypes.c_int64(0)
    idx = lib().kda_snapshot_lookup(_ptr(off), off.numel() - 1, int(seq), int(interval), int(prefix_len),
                                    ctypes.byref(cov))
    if idx == -2:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_snapshot_lookup")
    return int(idx), int(cov.value)


def kda_workspace_size(op: int, B: int, T: int, H: int, dk: int = 128, dv: int = 128, chunk: int = 64) -> int:
    return int(lib().kda_workspace_size(int(op), int(B), int(T), int(H), int(dk), int(dv), int(chunk)))


def kda_selftest_bounded_wait(stream=None) -> None:
    """Launch the bounded-wait diagnostic (about 2 s; afterwards the device status reads
    KDA_ERR_TIMEOUT)."""
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream(None)
    _check(lib().kda_selftest_bounded_wait(st), "kda_selftest_bounded_wait")


def kda_get_device_status(stream=None) -> int:
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream(None)
    return int(lib().kda_get_device_status(st))


def _workspace(op, B, T, H, dk, dv, chunk, device, workspace):
    need = kda_workspace_size(op, B, T, H, dk, dv, chunk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, (workspace.numel() * workspace.element_size() if workspace is not None else 0)


def _chunk(name, q, k, v, log_alpha, beta, init_state, out, final_state, chunk, out_dtype, return_final_state,
           workspace):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty(B, T, H, dv, dtype=out_dtype, device=q.device)
    if final_state is None and return_final_state:
        final_state = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    ws, ws_bytes = _workspace(KDA_OP_CHUNK, B, T, H, dk, dv, chunk, q.device, workspace)
    rc = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(init_state), _ptr(out),
                              _ptr(final_state), B, T, H, dk, dv, int(chunk), _dt(q), _dt(out), _ptr(ws), ws_bytes,
                              _stream(q.device))
    _check(rc, name)
    return out, final_state


def kda_chunk_fwd(q, k, v, log_alpha, beta, init_state=None, out=None, final_state=None, *, chunk: int = 64,
                  out_dtype=torch.float32, return_final_state: bool = True, workspace=None):
    """Batched prefill.  q,k [B,T,H,dk], v [B,T,H,dv] (bf16/fp32), log_alpha [B,T,H,dk] fp32,
    beta [B,T,H] fp32, init_state [B,H,dk,dv] fp32 or None.  Returns (out, final_state)."""
    return _chunk("kda_chunk_fwd", q, k, v, log_alpha, beta, init_state, out, final_state, chunk, out_dtype,
                  return_final_state, workspace)


def kda_chunk_fwd_host(q, k, v, log_alpha, beta, init_state=None, out=None, final_state=None, *,
                       out_dtype=torch.float32, segment_tokens: int = 0, workspace=None, device=None):
    """kda_chunk_fwd on HOST tensors (CPU; page-locked for overlap), streamed through the GPU
    in segments.  init_state is a device tensor or None; out and final_state are host tensors
    (allocated pinned if None).  Returns (out, final_state) once the call is enqueued on the
    current stream of `device` (cuda:0 by default); synchronise before reading them."""
    for t in (q, k, v, log_alpha, beta):
        if t.is_cuda:
            raise ValueError("kda_chunk_fwd_host takes host tensors")
    dev = torch.device(device or "cuda")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty(B, T, H, dv, dtype=out_dtype, pin_memory=True)
    if final_state is None:
        final_state = torch.empty(B, H, dk, dv, dtype=torch.float32, pin_memory=True)
    if workspace is None:
        need = lib().kda_host_fwd_workspace_size(B, H, dk, dv, int(segment_tokens), _dt(q), _dt(out))
        workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=dev)
    rc = lib().kda_chunk_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(init_state), _ptr(out),
                                  _ptr(final_state), B, T, H, dk, dv, _dt(q), _dt(out), int(segment_tokens),
                                  _ptr(workspace), workspace.numel(), _stream(dev))
    _check(rc, "kda_chunk_fwd_host")
    return out, final_state


def kda_gdn_chunk_fwd(q, k, v, log_alpha, beta, init_state=None, out=None, final_state=None, *, chunk: int = 64,
                      out_dtype=torch.float32, return_final_state: bool = True, workspace=None):
    """kda_chunk_fwd with one log-decay per (token, head): log_alpha [B,T,H] fp32 (Gated
    DeltaNet), or None for no decay (DeltaNet)."""
    return _chunk("kda_gdn_chunk_fwd", q, k, v, log_alpha, beta, init_state, out, final_state, chunk, out_dtype,
                  return_final_state, workspace)


def _varlen(name, q, k, v, log_alpha, beta, cu_seqlens, init_states, chunk, snapshot_interval, cu_seqlens_host,
            out, final_states, snapshots, out_dtype, workspace):
    Ttot, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty(Ttot, H, dv, dtype=out_dtype, device=q.device)
    if final_states is None:
        final_states = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
    snap_off = None
    if snapshot_interval:
        cu_h = cu_seqlens.cpu() if cu_seqlens_host is None else torch.as_tensor(cu_seqlens_host)
        off_h = kda_snapshot_offsets(cu_h, snapshot_interval)
        snap_off = off_h.to(q.device)
        if snapshots is None:
            snapshots = torch.empty(max(int(off_h[-1]), 1), H, dk, dv, dtype=torch.float32, device=q.device)
    ws, ws_bytes = _workspace(KDA_OP_VARLEN, N, Ttot, H, dk, dv, chunk, q.device, workspace)
    rc = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(cu_seqlens), N, Ttot,
                              H, dk, dv, int(chunk), _ptr(init_states), _ptr(final_states), int(snapshot_interval),
                              _ptr(snap_off), _ptr(snapshots) if snapshot_interval else None, _ptr(out), _dt(q),
                              _dt(out), _ptr(ws), ws_bytes, _stream(q.device))
    _check(rc, name)
    if snapshot_interval and snapshots is not None:
        snapshots = snapshots[: int(snap_off[-1].item())] if snapshots.shape[0] > 0 else snapshots
    return out, final_states, (snapshots if snapshot_interval else None)


def kda_varlen_fwd(q, k, v, log_alpha, beta, cu_seqlens, init_states=None, *, chunk: int = 64,
                   snapshot_interval: int = 0, cu_seqlens_host=None, out=None, final_states=None,
                   snapshots=None, out_dtype=torch.float32, workspace=None):
    """Packed sequences.  q,k [Ttot,H,dk], v [Ttot,H,dv], log_alpha [Ttot,H,dk], beta [Ttot,H];
    cu_seqlens int64 [N+1] on the device.  Returns (out, final_states, snapshots or None)."""
    return _varlen("kda_varlen_fwd", q, k, v, log_alpha, beta, cu_seqlens, init_states, chunk, snapshot_interval,
                   cu_seqlens_host, out, final_states, snapshots, out_dtype, workspace)


def kda_varlen_fwd_pool(q, k, v, log_alpha, beta, cu_seqlens, pool, init_slots=None, snap_slots=None, *,
                        gate: int = KDA_GATE_CHANNEL, chunk: int = 64, snapshot_interval: int = 0,
                        cu_seqlens_host=None, out=None, final_states=None, out_dtype=torch.float32, workspace=None):
    """Packed sequences over a state pool [pool_slots,H,dk,dv] (fp32, or bf16 storage with fp32
    arithmetic): sequence s starts from slot
    init_slots[s] (-1: zeros; None: all zeros) and snapshot m of sequence s goes to slot
    snap_slots[offsets[s] + m - 1] (-1: not stored).  log_alpha's layout is given by `gate`.
    Returns (out, final_states); the snapshots are in the pool."""
    Ttot, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty(Ttot, H, dv, dtype=out_dtype, device=q.device)
    if final_states is None:
        final_states = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
    if pool.dtype not in (torch.float32, torch.bfloat16) or tuple(pool.shape[1:]) != (H, dk, dv):
        raise ValueError(f"pool must be float32 or bfloat16 [slots, {H}, {dk}, {dv}]")
    snap_off = None
    if snapshot_interval:
        cu_h = cu_seqlens.cpu() if cu_seqlens_host is None else torch.as_tensor(cu_seqlens_host)
        snap_off = kda_snapshot_offsets(cu_h, snapshot_interval).to(q.device)
    for name, t in (("init_slots", init_slots), ("snap_slots", snap_slots)):
        if t is not None and t.dtype != torch.int64:
            raise TypeError(f"{name} must be int64")
    ws, ws_bytes = _workspace(KDA_OP_VARLEN, N, Ttot, H, dk, dv, chunk, q.device, workspace)
    rc = lib().kda_varlen_fwd_pool(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), int(gate), _ptr(beta),
                                   _ptr(cu_seqlens), N, Ttot, H, dk, dv, int(chunk), _ptr(pool), pool.shape[0],
                                   _dt(pool), _ptr(init_slots), int(snapshot_interval), _ptr(snap_off),
                                   _ptr(snap_slots),
                                   _ptr(final_states), _ptr(out), _dt(q), _dt(out), _ptr(ws), ws_bytes,
                                   _stream(q.device))
    _check(rc, "kda_varlen_fwd_pool")
    return out, final_states


def kda_gdn_varlen_fwd(q, k, v, log_alpha, beta, cu_seqlens, init_states=None, *, chunk: int = 64,
                       snapshot_interval: int = 0, cu_seqlens_host=None, out=None, final_states=None,
                       snapshots=None, out_dtype=torch.float32, workspace=None):
    """kda_varlen_fwd with log_alpha [Ttot,H] (Gated DeltaNet) or None (DeltaNet)."""
    return _varlen("kda_gdn_varlen_fwd", q, k, v, log_alpha, beta, cu_seqlens, init_states, chunk,
                   snapshot_interval, cu_seqlens_host, out, final_states, snapshots, out_dtype, workspace)


def _decode(fn, name, state_dtype, q, k, v, log_alpha, beta, state, out, out_dtype):
    if state.dtype != state_dtype:
        raise TypeError(f"{name}: state must be {state_dtype}, got {state.dtype}")
    B, H, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty(B, H, dv, dtype=out_dtype, device=q.device)
    rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(state), _ptr(out), B, H, dk, dv, _dt(q),
            _dt(out), _stream(q.device))
    _check(rc, name)
    return out


def kda_decode_step(q, k, v, log_alpha, beta, state, out=None, *, out_dtype=torch.float32):
    """One token per session: q,k [B,H,dk], v [B,H,dv], log_alpha [B,H,dk], beta [B,H];
    state [B,H,dk,dv] fp32 is updated in place.  Returns out [B,H,dv]."""
    return _decode(lib().kda_decode_step, "kda_decode_step", torch.float32, q, k, v, log_alpha, beta, state, out,
                   out_dtype)


def kda_decode_step_bf16state(q, k, v, log_alpha, beta, state, out=None, *, out_dtype=torch.float32):
    """kda_decode_step with a bf16-stored state [B,H,dk,dv] (updated in place; the step
    itself runs in fp32 and the output is read before the state is rounded)."""
    return _decode(lib().kda_decode_step_bf16state, "kda_decode_step_bf16state", torch.bfloat16, q, k, v, log_alpha,
                   beta, state, out, out_dtype)


def kda_gdn_decode_step_bf16state(q, k, v, log_alpha, beta, state, out=None, *, out_dtype=torch.float32):
    """kda_gdn_decode_step with a bf16-stored state (fp32 arithmetic)."""
    return _decode(lib().kda_gdn_decode_step_bf16state, "kda_gdn_decode_step_bf16state", torch.bfloat16, q, k, v,
                   log_alpha, beta, state, out, out_dtype)


def kda_gdn_decode_step(q, k, v, log_alpha, beta, state, out=None, *, out_dtype=torch.float32):
    """kda_decode_step with log_alpha [B,H] (Gated DeltaNet) or None (DeltaNet); fp32 state."""
    return _decode(lib().kda_gdn_decode_step, "kda_gdn_decode_step", torch.float32, q, k, v, log_alpha, beta, state,
                   out, out_dtype)


def kda_bwd(q, k, v, log_alpha, beta, d_out, init_state=None, d_final_state=None, *, gate: int = KDA_GATE_CHANNEL,
            cu_seqlens=None, return_d_init: bool = True, chunk: int = 64, workspace=None,
            no_alloc: bool = False) -> dict:
    """Gradients of L = sum <d_out, o> + <d_final_state, S_final> through the forward of
    kda_chunk_fwd (batched q [B,T,H,dk] when cu_seqlens is None, else packed [Ttot,H,dk]).
    log_alpha's layout follows `gate`.  Returns dict(dq, dk, dv, dlog_alpha, dbeta, d_init).
    chunk=64 calls kda_chunk_bwd (chunked), chunk=1 the token-serial kda_bwd; no_alloc=True
    calls kda_bwd_noalloc (token-serial, the library's static scratch, no workspace)."""
    if cu_seqlens is None:
        N, T, H, dk = q.shape
        t_arg, t_total = T, N * T
    else:
        t_total, H, dk = q.shape
        N = cu_seqlens.numel() - 1
        t_arg = t_total
    dv = v.shape[-1]
    f32 = dict(dtype=torch.float32, device=q.device)
    g = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(k.shape, **f32), "dv": torch.empty(v.shape, **f32),
         "dlog_alpha": None if gate == KDA_GATE_NONE else torch.empty(log_alpha.shape, **f32),
         "dbeta": torch.empty(beta.shape, **f32),
         "d_init": torch.empty(N, H, dk, dv, **f32) if return_d_init else None}
    head = (_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), int(gate), _ptr(beta), _ptr(init_state), _ptr(d_out),
            _ptr(d_final_state), _ptr(cu_seqlens), N, t_arg, H, dk, dv)
    grads = (_ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_alpha"]), _ptr(g["dbeta"]),
             _ptr(g["d_init"]), _dt(q))
    if no_alloc:
        _check(lib().kda_bwd_noalloc(*head, *grads, _stream(q.device)), "kda_bwd_noalloc")
        return g
    if workspace is None:
        need = kda_workspace_size(KDA_OP_CHUNK_BWD, N, t_total, H, dk, dv, chunk)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if chunk == 1:
        rc, name = lib().kda_bwd(*head, *grads, _ptr(workspace), workspace.numel(), _stream(q.device)), "kda_bwd"
    else:
        rc = lib().kda_chunk_bwd(*head, int(chunk), *grads, _ptr(workspace), workspace.numel(), _stream(q.device))
        name = "kda_chunk_bwd"
    _check(rc, name)
    return g


# ---------------------------------------------------------------- operators around the recurrence
_CODE = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}


def _code(dtype, what: str) -> int:
    try:
        return _CODE[dtype]
    except KeyError:
        raise TypeError(f"{what}: unsupported dtype {dtype}, use bfloat16 or float32") from None


def _addr(t):
    return None if t is None else t.data_ptr()


def _full(t, name: str, shape, dtype, dev: int):
    """A contiguous tensor (or None) of this shape and dtype on device `dev`; its address."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {list(shape)}, got {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name: str, lead, row, dtype, dev: int) -> int:
    """Checks a tensor of rows [*lead, *row]: a row contiguous, the rows equally far apart.  Returns that
    distance in elements."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (*lead, *row):
        raise ValueError(f"{name} must have the shape {[*lead, *row]}, got {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    n = 1
    for x in row:
        n *= x
    if t.is_contiguous():
        return n
    shape, stride = t.shape, t.stride()
    want, at = 1, len(shape) - 1
    while at >= len(lead):  # the row itself
        if shape[at] != 1 and stride[at] != want:
            raise ValueError(f"{name}: every row must be contiguous")
        want *= shape[at]
        at -= 1
    step = None
    for i in range(at, -1, -1):  # the rows, from the innermost dimension
        if shape[i] != 1:
            if step is None:
                step, unit = stride[i], stride[i]
            elif stride[i] != unit:
                raise ValueError(f"{name}: the rows must be equally far apart")
            unit *= shape[i]
    if step is not None and step < n:
        raise ValueError(f"{name}: the rows must not overlap")
    return n if step is None else step


def _on_gpu(t, name: str) -> int:
    """The tensor's device, as its number."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    _same_device(dev, f"{name} is on")
    return dev


# The handle of a device's current stream; the plain accessor builds a Stream object around it each time.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _sequences(lead, cu_seqlens, dev: int):
    """(address of cu_seqlens, N, T as the C call wants it, T_total) for activations [*lead, ..]."""
    if cu_seqlens is None:
        if len(lead) != 2:
            raise ValueError("activations must be [B, T, ..] without cu_seqlens and [T_total, ..] with it")
        return None, lead[0], lead[1], lead[0] * lead[1]
    if len(lead) != 1:
        raise ValueError("activations must be [T_total, ..] with cu_seqlens")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N + 1]")
    return _full(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int64, dev), cu_seqlens.numel() - 1, lead[0], lead[0]


def _scratch(need: int, workspace, like):
    """The caller's workspace, or a new one; (tensor, address, bytes)."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty((need,), dtype=torch.uint8, device=like.device)
    elif not workspace.is_contiguous() or workspace.get_device() != like.get_device():
        raise ValueError("workspace must be contiguous and on the inputs' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _conv_args(x, weight, bias, lead, device: int):
    D = x.shape[-1]
    if weight.dim() != 2:
        raise ValueError("weight must be [D, width]")
    W = weight.shape[1]
    f32 = torch.float32
    return (D, W, _rows(x, "x", lead, (D,), x.dtype, device), _full(weight, "weight", (D, W), f32, device),
            _full(bias, "bias", (D,), f32, device))


def kda_conv_fwd(x, weight, bias=None, init_state=None, out=None, final_state=None, *, cu_seqlens=None,
                 activation: int = KDA_ACT_SILU, out_dtype=None, return_final_state: bool = True):
    """Short causal convolution over each channel.  x [B,T,D], or [Ttot,D] with cu_seqlens (int64 [N+1]); a slice
    of a wider tensor's last dimension is read in place.  weight [D,W] fp32 (W = 2, 3, 4), bias [D] fp32 or None,
    init_state [N,W-1,D] in x's dtype or None (zeros).  Returns (out, final_state); a new out has out_dtype
    (x's dtype by default), a given one keeps its own.  final_state may be init_state itself."""
    dev, lead = _on_gpu(x, "x"), x.shape[:-1]
    cu, N, T, _ = _sequences(lead, cu_seqlens, dev)
    D, W, xs, w, b = _conv_args(x, weight, bias, lead, dev)
    if out is None:
        out = torch.empty((*lead, D), dtype=out_dtype or x.dtype, device=x.device)
    if final_state is None and return_final_state:
        final_state = torch.empty((N, W - 1, D), dtype=x.dtype, device=x.device)
    _check(lib().kda_conv_fwd(x.data_ptr(), xs, w, b, _full(init_state, "init_state", (N, W - 1, D), x.dtype, dev),
                              _full(out, "out", (*lead, D), out.dtype, dev),
                              _full(final_state, "final_state", (N, W - 1, D), x.dtype, dev), cu, N, T, D, W,
                              activation, _code(x.dtype, "x"), _code(out.dtype, "out"), _raw_stream(dev)), "kda_conv_fwd")
    return out, final_state


def kda_conv_step(x, weight, bias, state, out=None, *, activation: int = KDA_ACT_SILU, out_dtype=None):
    """kda_conv_fwd for one token per session: x [B,D]; state [B,W-1,D] in x's dtype is moved on in place.
    Returns out [B,D]."""
    dev = _on_gpu(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [B, D]")
    D, W, xs, w, b = _conv_args(x, weight, bias, x.shape[:-1], dev)
    B = x.shape[0]
    if out is None:
        out = torch.empty((B, D), dtype=out_dtype or x.dtype, device=x.device)
    _check(lib().kda_conv_step(x.data_ptr(), xs, w, b, _full(state, "state", (B, W - 1, D), x.dtype, dev),
                               _full(out, "out", (B, D), out.dtype, dev), B, D, W, activation, _code(x.dtype, "x"),
                               _code(out.dtype, "out"), _raw_stream(dev)), "kda_conv_step")
    return out


def kda_conv_bwd(x, weight, bias, d_out, init_state=None, d_final_state=None, *, cu_seqlens=None,
                 activation: int = KDA_ACT_SILU, return_d_init: bool = True, workspace=None) -> dict:
    """Gradients of sum <d_out, out> (+ sum <d_final_state, final_state>) through kda_conv_fwd.  Returns dict(dx in
    d_out's dtype; dweight, dbias (None without a bias) and d_init (None without an init_state) fp32)."""
    dev, lead = _on_gpu(x, "x"), x.shape[:-1]
    cu, N, T, total = _sequences(lead, cu_seqlens, dev)
    D, W, xs, w, b = _conv_args(x, weight, bias, lead, dev)
    f32 = dict(dtype=torch.float32, device=x.device)
    g = {"dx": torch.empty((*lead, D), dtype=d_out.dtype, device=x.device), "dweight": torch.empty((D, W), **f32),
         "dbias": None if bias is None else torch.empty((D,), **f32),
         "d_init": torch.empty((N, W - 1, D), **f32) if init_state is not None and return_d_init else None}
    ws, wp, wb = _scratch(lib().kda_conv_bwd_workspace_size(total, D, W), workspace, x)
    _check(lib().kda_conv_bwd(x.data_ptr(), xs, w, b, _full(init_state, "init_state", (N, W - 1, D), x.dtype, dev),
                              _full(d_out, "d_out", (*lead, D), d_out.dtype, dev),
                              _full(d_final_state, "d_final_state", (N, W - 1, D), torch.float32, dev), cu, N, T, D,
                              W, activation, _addr(g["dx"]), _addr(g["dweight"]), _addr(g["dbias"]),
                              _addr(g["d_init"]), _code(x.dtype, "x"), _code(d_out.dtype, "d_out"), wp, wb,
                              _raw_stream(dev)), "kda_conv_bwd")
    return g


def _ssm_args(u, delta, A, B, C, D, z, delta_bias, delta_softplus, lead, dev):
    """The common head of the scan's calls, and (D, n_state, G)."""
    Dm, dt, f32 = u.shape[-1], u.dtype, torch.float32
    if A.dim() != 2 or B.dim() != len(lead) + 2:
        raise ValueError("A must be [D, n_state], B and C [.., G, n_state]")
    G, N = B.shape[-2:]
    head = (u.data_ptr(), _rows(u, "u", lead, (Dm,), dt, dev), delta.data_ptr(),
            _rows(delta, "delta", lead, (Dm,), dt, dev), _full(A, "A", (Dm, N), f32, dev), B.data_ptr(),
            _rows(B, "B", lead, (G, N), dt, dev), C.data_ptr(), _rows(C, "C", lead, (G, N), dt, dev),
            _full(D, "D", (Dm,), f32, dev), _addr(z), 0 if z is None else _rows(z, "z", lead, (Dm,), dt, dev),
            _full(delta_bias, "delta_bias", (Dm,), f32, dev), int(bool(delta_softplus)))
    return head, (Dm, N, G)


def kda_ssm_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, init_state=None, out=None, final_state=None, *,
                cu_seqlens=None, delta_softplus: bool = True, out_dtype=None, return_final_state: bool = True,
                workspace=None):
    """Selective state space scan.  u, delta (and the gate z) [B,T,D], or [Ttot,D] with cu_seqlens; B, C [..,G,n]
    with G dividing D, all in u's dtype, slices of wider tensors read in place; A [D,n] fp32 (n <= 64), D and
    delta_bias [D] fp32 or None, init_state [N,D,n] fp32 or None.  Returns (out, final_state [N,D,n] fp32); a new out
    has out_dtype (u's dtype by default), a given one keeps its own."""
    dev, lead = _on_gpu(u, "u"), u.shape[:-1]
    cu, N, T, total = _sequences(lead, cu_seqlens, dev)
    head, (Dm, n, G) = _ssm_args(u, delta, A, B, C, D, z, delta_bias, delta_softplus, lead, dev)
    if out is None:
        out = torch.empty((*lead, Dm), dtype=out_dtype or u.dtype, device=u.device)
    if final_state is None and return_final_state:
        final_state = torch.empty((N, Dm, n), dtype=torch.float32, device=u.device)
    ws, wp, wb = _scratch(lib().kda_ssm_fwd_workspace_size(N, total, Dm, n, G, cu is not None), workspace, u)
    _check(lib().kda_ssm_fwd(*head, _full(init_state, "init_state", (N, Dm, n), torch.float32, dev),
                             _full(out, "out", (*lead, Dm), out.dtype, dev),
                             _full(final_state, "final_state", (N, Dm, n), torch.float32, dev), cu, N, T, Dm, n, G,
                             _code(u.dtype, "u"), _code(out.dtype, "out"), wp, wb, _raw_stream(dev)), "kda_ssm_fwd")
    return out, final_state


def kda_ssm_step(u, delta, A, B, C, D, z, delta_bias, state, out=None, *, delta_softplus: bool = True,
                 out_dtype=None):
    """kda_ssm_fwd for one token per session: u, delta, z [S,D], B, C [S,G,n]; state [S,D,n] fp32 is updated in
    place.  Returns out [S,D]."""
    dev, lead = _on_gpu(u, "u"), u.shape[:-1]
    if len(lead) != 1:
        raise ValueError("u must be [S, D]")
    head, (Dm, n, G) = _ssm_args(u, delta, A, B, C, D, z, delta_bias, delta_softplus, lead, dev)
    S = lead[0]
    if out is None:
        out = torch.empty((S, Dm), dtype=out_dtype or u.dtype, device=u.device)
    _check(lib().kda_ssm_step(*head, _full(state, "state", (S, Dm, n), torch.float32, dev),
                              _full(out, "out", (S, Dm), out.dtype, dev), S, Dm, n, G, _code(u.dtype, "u"),
                              _code(out.dtype, "out"), _raw_stream(dev)), "kda_ssm_step")
    return out


def kda_ssm_bwd(u, delta, A, B, C, d_out, D=None, z=None, delta_bias=None, init_state=None, d_final_state=None, *,
                cu_seqlens=None, delta_softplus: bool = True, return_d_init: bool = True, workspace=None) -> dict:
    """Gradients of sum <d_out, out> (+ sum <d_final_state, final_state>) through kda_ssm_fwd.  Returns dict(du,
    ddelta, dz in d_out's dtype; dA, dB, dC, dD, ddelta_bias, d_init fp32), None for inputs that were None."""
    dev, lead = _on_gpu(u, "u"), u.shape[:-1]
    cu, N, T, total = _sequences(lead, cu_seqlens, dev)
    head, (Dm, n, G) = _ssm_args(u, delta, A, B, C, D, z, delta_bias, delta_softplus, lead, dev)
    f32, act = dict(dtype=torch.float32, device=u.device), dict(dtype=d_out.dtype, device=u.device)
    new = torch.empty
    g = {"du": new((*lead, Dm), **act), "ddelta": new((*lead, Dm), **act), "dA": new((Dm, n), **f32),
         "dB": new((*lead, G, n), **f32), "dC": new((*lead, G, n), **f32),
         "dD": None if D is None else new((Dm,), **f32), "dz": None if z is None else new((*lead, Dm), **act),
         "ddelta_bias": None if delta_bias is None else new((Dm,), **f32),
         "d_init": new((N, Dm, n), **f32) if init_state is not None and return_d_init else None}
    ws, wp, wb = _scratch(lib().kda_ssm_bwd_workspace_size(N, total, Dm, n, G, cu is not None), workspace, u)
    _check(lib().kda_ssm_bwd(*head, _full(init_state, "init_state", (N, Dm, n), torch.float32, dev),
                             _full(d_out, "d_out", (*lead, Dm), d_out.dtype, dev),
                             _full(d_final_state, "d_final_state", (N, Dm, n), torch.float32, dev), cu, N, T, Dm, n, G,
                             *(_addr(g[k]) for k in ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias",
                                                     "d_init")),
                             _code(u.dtype, "u"), _code(d_out.dtype, "d_out"), wp, wb, _raw_stream(dev)), "kda_ssm_bwd")
    return g


def _head_args(q, k, q_weight, k_weight, cos, sin, positions, dev):
    """(lead, tokens, Hq, Hk, d, rot) and the addresses and strides of the inputs."""
    if q.dim() < 3:
        raise ValueError("q must be [.., H, d]")
    lead, (Hq, d) = q.shape[:-2], q.shape[-2:]
    tokens = 1
    for x in lead:
        tokens *= x
    Hk = 0 if k is None else k.shape[-2]
    ptrs = [q.data_ptr(), _rows(q, "q", lead, (Hq, d), q.dtype, dev), _addr(k),
            0 if k is None else _rows(k, "k", lead, (Hk, d), q.dtype, dev)]
    f32 = torch.float32
    weights = [_full(q_weight, "q_weight", (d,), f32, dev), _full(k_weight, "k_weight", (d,), f32, dev)]
    rot, tables = 0, [None, None, None, 0]
    if cos is not None or sin is not None:  # positions alone turn nothing
        if cos is None or sin is None or positions is None or cos.dim() != 2:
            raise ValueError("the rotation wants cos and sin [positions, rot / 2] and positions")
        rot = 2 * cos.shape[1]
        tables = [_full(cos, "cos", cos.shape, f32, dev), _full(sin, "sin", cos.shape, f32, dev),
                  _full(positions, "positions", lead, torch.int64, dev), cos.shape[0]]
    return (lead, tokens, Hq, Hk, d, rot), ptrs, weights, tables


def kda_qk_norm_fwd(q, k=None, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, *,
                    norm: int = KDA_NORM_L2, layout: int = KDA_ROT_HALF, eps: float = 1e-6, q_out=None, k_out=None,
                    out_dtype=None):
    """Norm of every query and key head with the position rotation in the same pass.  q [..,Hq,d], k [..,Hk,d] or
    None (slices of wider tensors are read in place), weights [d] fp32 or None; cos, sin [P, rot/2] fp32 and
    positions [..] int64 turn the first rot channels (cos and sin None: no rotation, whatever the positions).  Returns
    (q_out, k_out); new ones have out_dtype (q's dtype by default), given ones share a dtype."""
    dev = _on_gpu(q, "q")
    (lead, tokens, Hq, Hk, d, rot), ptrs, weights, tables = _head_args(q, k, q_weight, k_weight, cos, sin, positions, dev)
    if q_out is None:
        q_out = torch.empty((*lead, Hq, d), dtype=out_dtype or q.dtype, device=q.device)
    if k_out is None and k is not None:
        k_out = torch.empty((*lead, Hk, d), dtype=q_out.dtype, device=q.device)
    _check(lib().kda_qk_norm_fwd(*ptrs, *weights, *tables, _full(q_out, "q_out", (*lead, Hq, d), q_out.dtype, dev),
                                 _full(k_out, "k_out", (*lead, Hk, d), q_out.dtype, dev), tokens, Hq, Hk, d, rot,
                                 layout, norm, eps, _code(q.dtype, "q"), _code(q_out.dtype, "q_out"), _raw_stream(dev)),
           "kda_qk_norm_fwd")
    return q_out, k_out


def kda_qk_norm_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, *,
                    norm: int = KDA_NORM_L2, layout: int = KDA_ROT_HALF, eps: float = 1e-6, workspace=None) -> dict:
    """Gradients of sum <dq_out, q_out> + <dk_out, k_out> through kda_qk_norm_fwd.  Returns dict(dq, dk in dq_out's
    dtype; dq_weight, dk_weight fp32), None for inputs that were None."""
    dev = _on_gpu(q, "q")
    (lead, tokens, Hq, Hk, d, rot), ptrs, weights, tables = _head_args(q, k, q_weight, k_weight, cos, sin, positions, dev)
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    act, f32 = dict(dtype=dq_out.dtype, device=q.device), dict(dtype=torch.float32, device=q.device)
    g = {"dq": torch.empty((*lead, Hq, d), **act), "dk": None if k is None else torch.empty((*lead, Hk, d), **act),
         "dq_weight": None if q_weight is None else torch.empty((d,), **f32),
         "dk_weight": None if k_weight is None else torch.empty((d,), **f32)}
    need = 0 if q_weight is None and k_weight is None else lib().kda_qk_norm_bwd_workspace_size(d)
    ws, wp, wb = _scratch(need, workspace, q)
    _check(lib().kda_qk_norm_bwd(*ptrs, _full(dq_out, "dq_out", (*lead, Hq, d), dq_out.dtype, dev),
                                 _full(dk_out, "dk_out", (*lead, Hk, d), dq_out.dtype, dev), *weights, *tables,
                                 _addr(g["dq"]), _addr(g["dk"]), _addr(g["dq_weight"]), _addr(g["dk_weight"]), tokens,
                                 Hq, Hk, d, rot, layout, norm, eps, _code(q.dtype, "q"),
                                 _code(dq_out.dtype, "dq_out"), wp, wb, _raw_stream(dev)), "kda_qk_norm_bwd")
    return g
