"""GB300-native LM-head contraction fused with the consumer-surface projection.

Thin ctypes binding over the C ABI in ``include/sb.h`` (``libsb.so``, built in-tree by
``gemm_epilogue_reduction_gb300.build``). The functions named ``sb_*`` mirror the C entry
points one to one and only marshal arguments: every step of the path runs in the CUDA
kernels. ``project`` is a convenience wrapper that allocates the outputs and workspace with
torch (the caller-owned memory of the C ABI) and raises on a non-OK status.

There is no CPU fallback: if ``libsb.so`` is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

SB_TOKEN, SB_TOKEN_LOGPROB, SB_FULL_LOGITS, SB_GUMBEL_TOKEN, SB_TOPK_LOGPROB = 0, 1, 2, 3, 4
SB_MAX_TOPK = 16
SB_W_PACKED = 0x100  # layout flag OR'ed into `surface`: W is the packed copy (sb_pack_weights)
SURFACES = {"token": SB_TOKEN, "token_logprob": SB_TOKEN_LOGPROB,
            "full_logits": SB_FULL_LOGITS, "gumbel_token": SB_GUMBEL_TOKEN,
            "topk_logprob": SB_TOPK_LOGPROB}
SB_REDUCE_NONE, SB_REDUCE_SUM, SB_REDUCE_MEAN = 0, 1, 2
SB_BF16, SB_F32 = 0, 1
SB_GATE_NONE, SB_GATE_CHANNEL, SB_GATE_TOKEN = 0, 1, 2
REDUCTIONS = {"none": SB_REDUCE_NONE, "sum": SB_REDUCE_SUM, "mean": SB_REDUCE_MEAN}
SB_OK = 0
SB_ERR_INVALID_ARG = 1
SB_ERR_UNSUPPORTED = 2
SB_ERR_ALIGNMENT = 3
SB_ERR_WORKSPACE_TOO_SMALL = 4
SB_ERR_CUDA = 5
SB_ERR_DEVICE_TIMEOUT = 6

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libsb.so")
_lock = threading.Lock()
_lib = None


class SbError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: status {status} ({sb_status_string(status)})")
        self.status = status


class sb_outputs(ctypes.Structure):
    _fields_ = [("token", ctypes.c_void_p), ("token_logprob", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("logits_bf16", ctypes.c_void_p),
                ("target_ids", ctypes.c_void_p), ("target_logprob", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("topk_ids", ctypes.c_void_p), ("topk_logprob", ctypes.c_void_p),
                ("topk", ctypes.c_int32)]


class sb_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("scale_sq", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("weight_decay", ctypes.c_double), ("param_type", ctypes.c_int32),
                ("grad_type", ctypes.c_int32)]


def lib():
    """The loaded libsb.so; raises if it has not been built."""
    global _lib
    L = _lib
    if L is not None:  # the common case: no lock once loaded
        return L
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libsb.so not found at {LIB_PATH}: build it first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        P, i64, i32, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64
        L.sb_workspace_bytes.argtypes = [i64, i64, i32, i32]
        L.sb_workspace_bytes.restype = ctypes.c_size_t
        L.sb_tiles_per_shard.argtypes = [i64, i64, i32]
        L.sb_tiles_per_shard.restype = i32
        L.sb_packed_weight_bytes.argtypes = [i64, i64, i32]
        L.sb_packed_weight_bytes.restype = ctypes.c_size_t
        L.sb_pack_weights.argtypes = [P, i64, i64, i32, P, ctypes.c_size_t, P]
        L.sb_pack_weights.restype = i32
        L.sb_lmhead_project.argtypes = [P, P, i64, i64, i64, i32, i32, ctypes.c_float, u64,
                                        ctypes.POINTER(sb_outputs), P]
        L.sb_lmhead_project.restype = i32
        L.sb_lmhead_records.argtypes = L.sb_lmhead_project.argtypes
        L.sb_lmhead_records.restype = i32
        L.sb_lmhead_project_static_scratch.argtypes = L.sb_lmhead_project.argtypes
        L.sb_lmhead_project_static_scratch.restype = i32
        L.sb_static_scratch_last_status.argtypes = []
        L.sb_static_scratch_last_status.restype = i32
        L.sb_lmhead_project_from_host.argtypes = [P, P, P, i64, i64, i64, i32, i32,
                                                  ctypes.c_float, u64,
                                                  ctypes.POINTER(sb_outputs), P, P, P]
        L.sb_lmhead_project_from_host.restype = i32
        L.sb_host_step_create.argtypes = [P, P, P, i64, i64, i64, i32, i32, ctypes.c_float,
                                          u64, ctypes.POINTER(sb_outputs), P, P,
                                          ctypes.POINTER(P)]
        L.sb_host_step_create.restype = i32
        L.sb_host_step_launch.argtypes = [P, P]
        L.sb_host_step_launch.restype = i32
        L.sb_host_step_destroy.argtypes = [P]
        L.sb_host_step_destroy.restype = None
        L.sb_combine_shard_records.argtypes = [P, i64, i32, i32, i32, ctypes.c_float,
                                               ctypes.POINTER(sb_outputs), P]
        L.sb_combine_shard_records.restype = i32
        L.sb_payload_bytes.argtypes = [i64, i32, i32]
        L.sb_payload_bytes.restype = ctypes.c_size_t
        L.sb_pack_shard_records.argtypes = [P, i64, i32, i32, i32, i64, P, P]
        L.sb_pack_shard_records.restype = i32
        L.sb_merge_shard_payload.argtypes = [P, i64, i32, i32, ctypes.c_float,
                                             ctypes.POINTER(sb_outputs), P]
        L.sb_merge_shard_payload.restype = i32
        L.sb_partial_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.sb_partial_workspace_bytes.restype = ctypes.c_size_t
        L.sb_partial_completion.argtypes = [P, P, i64, i64, i64, i32, P, i32, P,
                                            ctypes.c_size_t, P]
        L.sb_partial_completion.restype = i32
        L.sb_debug_map_encodes.argtypes = []
        L.sb_debug_map_encodes.restype = ctypes.c_uint64
        L.sb_cross_entropy_workspace_bytes.argtypes = [i64] * 3
        L.sb_cross_entropy_workspace_bytes.restype = ctypes.c_size_t
        L.sb_cross_entropy_forward.argtypes = [P, P, P, i64, i64, i64, i32, i32, ctypes.c_float,
                                               P, P, P, ctypes.c_size_t, P]
        L.sb_cross_entropy_forward.restype = i32
        L.sb_cross_entropy_backward_workspace_bytes.argtypes = [i64] * 4 + [i32] * 2
        L.sb_cross_entropy_backward_workspace_bytes.restype = ctypes.c_size_t
        L.sb_cross_entropy_backward.argtypes = [P, P, P, P, P, i64, i64, i64, i32, i32,
                                                ctypes.c_float, i64, P, P, P, ctypes.c_size_t, P]
        L.sb_cross_entropy_backward.restype = i32
        f32, f64 = ctypes.c_float, ctypes.c_double
        L.sb_residual_norm_forward.argtypes = [P] * 5 + [i32, i64, i64, i32, i32, f32, f32, P, P, P]
        L.sb_residual_norm_forward.restype = i32
        L.sb_residual_norm_workspace_bytes.argtypes = [i64] * 2
        L.sb_residual_norm_workspace_bytes.restype = ctypes.c_size_t
        L.sb_residual_norm_backward.argtypes = ([P] * 7 + [i32, i64, i64, i32, i32, f32, f32] +
                                                [P] * 6 + [ctypes.c_size_t, P])
        L.sb_residual_norm_backward.restype = i32
        L.sb_adamw_step.argtypes = [P, i64, f64, f64, f64, f64, i64, i32, P, P]
        L.sb_adamw_step.restype = i32
        L.sb_select_source_projection.argtypes = [ctypes.c_double] * 8 + [
            ctypes.POINTER(ctypes.c_double)]
        L.sb_select_source_projection.restype = i32
        L.sb_last_device_status.argtypes = [ctypes.POINTER(sb_outputs)]
        L.sb_last_device_status.restype = i32
        L.sb_status_string.argtypes = [i32]
        L.sb_status_string.restype = ctypes.c_char_p
        L.sb_device_info.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.sb_device_info.restype = i32
        L.sb_debug_combine_math.argtypes = [i32, P, P, i64, P]
        L.sb_debug_combine_math.restype = i32
        L.sb_debug_gumbel_from_bits.argtypes = [P, P, i64, P]
        L.sb_debug_gumbel_from_bits.restype = i32
        L.sb_debug_configure.argtypes = [i32, u64]
        L.sb_debug_configure.restype = i32
        _lib = L
        return L


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        if torch.cuda.is_initialized():
            return _current(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


# ------------------------------------------------------------------ C entry points
def sb_workspace_bytes(M: int, V: int, k: int, surface: int) -> int:
    return int(lib().sb_workspace_bytes(M, V, k, surface))


def sb_tiles_per_shard(M: int, V: int, k: int) -> int:
    return int(lib().sb_tiles_per_shard(M, V, k))


def sb_packed_weight_bytes(V: int, d: int, k: int) -> int:
    return int(lib().sb_packed_weight_bytes(V, d, k))


def sb_pack_weights(W, V, d, k, W_packed, nbytes, stream=None) -> int:
    return int(lib().sb_pack_weights(_ptr(W), V, d, k, _ptr(W_packed), nbytes,
                                     _stream(stream)))


def sb_lmhead_project(H, W, M, d, V, k, surface, temperature, seed, out: sb_outputs,
                      stream=None) -> int:
    return int(lib().sb_lmhead_project(_ptr(H), _ptr(W), M, d, V, k, surface,
                                       float(temperature), seed & (2**64 - 1),
                                       ctypes.byref(out), _stream(stream)))


def sb_lmhead_project_from_host(H_host, H_dev, W, M, d, V, k, surface, temperature, seed,
                                out: sb_outputs, token_host, token_logprob_host=None,
                                stream=None) -> int:
    """H_host, token_host and token_logprob_host are host tensors (pinned for asynchronous
    copies) or raw host addresses; H_dev and W are device tensors."""
    return int(lib().sb_lmhead_project_from_host(
        _ptr(H_host), _ptr(H_dev), _ptr(W), M, d, V, k, surface, float(temperature),
        seed & (2**64 - 1), ctypes.byref(out), _ptr(token_host), _ptr(token_logprob_host),
        _stream(stream)))


def sb_host_step_create(H_host, H_dev, W, M, d, V, k, surface, temperature, seed,
                        out: sb_outputs, token_host, token_logprob_host=None):
    """Returns (status, handle); the handle is an int (0 on error)."""
    h = ctypes.c_void_p()
    st = int(lib().sb_host_step_create(
        _ptr(H_host), _ptr(H_dev), _ptr(W), M, d, V, k, surface, float(temperature),
        seed & (2**64 - 1), ctypes.byref(out), _ptr(token_host), _ptr(token_logprob_host),
        ctypes.byref(h)))
    return st, (h.value or 0)


def sb_host_step_launch(step: int, stream=None) -> int:
    return int(lib().sb_host_step_launch(step, _stream(stream)))


def sb_host_step_destroy(step: int) -> None:
    lib().sb_host_step_destroy(step)


class HostStep:
    """A host-buffer decode step captured once (sb_host_step_*): call it to enqueue one
    replay; the buffers passed here are read and written by every replay, so the caller
    keeps them alive and pinned."""

    def __init__(self, H_host, H_dev, W, M, d, V, k, surface, temperature, seed,
                 out: sb_outputs, token_host, token_logprob_host=None):
        self._keep = (H_host, H_dev, W, out, token_host, token_logprob_host)
        st, self.handle = sb_host_step_create(H_host, H_dev, W, M, d, V, k, surface,
                                              temperature, seed, out, token_host,
                                              token_logprob_host)
        if st != SB_OK:
            raise SbError(st, "sb_host_step_create")

    def __call__(self, stream=None) -> None:
        st = sb_host_step_launch(self.handle, stream)
        if st != SB_OK:
            raise SbError(st, "sb_host_step_launch")

    def close(self) -> None:
        if self.handle:
            sb_host_step_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sb_lmhead_records(H, W, M, d, V, k, surface, temperature, seed, out: sb_outputs,
                      stream=None) -> int:
    return int(lib().sb_lmhead_records(_ptr(H), _ptr(W), M, d, V, k, surface,
                                       float(temperature), seed & (2**64 - 1),
                                       ctypes.byref(out), _stream(stream)))


def sb_lmhead_project_static_scratch(H, W, M, d, V, k, surface, temperature, seed,
                                     out: sb_outputs, stream=None) -> int:
    """sb_lmhead_project with the library's built-in 8 MiB scratch instead of
    out.workspace, for callers that cannot allocate device memory."""
    return int(lib().sb_lmhead_project_static_scratch(_ptr(H), _ptr(W), M, d, V, k, surface,
                                                      float(temperature), seed & (2**64 - 1),
                                                      ctypes.byref(out), _stream(stream)))


def sb_static_scratch_last_status() -> int:
    """Device status of the last static-scratch call on the current device (synchronises)."""
    return int(lib().sb_static_scratch_last_status())


def sb_combine_shard_records(workspace, M, k, tiles_per_shard, surface, temperature,
                             out: sb_outputs, stream=None) -> int:
    return int(lib().sb_combine_shard_records(_ptr(workspace), M, k, tiles_per_shard,
                                              surface, float(temperature),
                                              ctypes.byref(out), _stream(stream)))


def sb_payload_bytes(M: int, k: int, surface: int) -> int:
    return int(lib().sb_payload_bytes(M, k, surface))


def sb_pack_shard_records(workspace, M, k, tiles_per_shard, surface, col_offset, payload,
                          stream=None) -> int:
    return int(lib().sb_pack_shard_records(_ptr(workspace), M, k, tiles_per_shard, surface,
                                           int(col_offset), _ptr(payload), _stream(stream)))


def sb_merge_shard_payload(payload, M, k, surface, temperature, out: sb_outputs,
                           stream=None) -> int:
    return int(lib().sb_merge_shard_payload(_ptr(payload), M, k, surface, float(temperature),
                                            ctypes.byref(out), _stream(stream)))


def sb_partial_workspace_bytes(M: int, N: int, K: int, lanes: int) -> int:
    return int(lib().sb_partial_workspace_bytes(M, N, K, lanes))


def sb_partial_completion(X, W, M, N, K, lanes, Y, y_bf16, workspace, workspace_bytes,
                          stream=None) -> int:
    return int(lib().sb_partial_completion(_ptr(X), _ptr(W), M, N, K, lanes, _ptr(Y),
                                           1 if y_bf16 else 0, _ptr(workspace),
                                           int(workspace_bytes), _stream(stream)))


def partial_completion(X, W, lanes: int, *, out_bf16: bool = True, stream=None, workspace=None):
    """Y = sum over lanes of X[:, lane] W[:, lane]^T for torch CUDA bf16 tensors X [M, K] and
    W [N, K]; returns (Y, workspace).  Raises SbError on a bad status."""
    import torch
    M, K = X.shape
    N = W.shape[0]
    nbytes = sb_partial_workspace_bytes(M, N, K, lanes)
    if nbytes == 0:
        raise SbError(SB_ERR_INVALID_ARG, "sb_partial_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    Y = torch.empty(M, N, dtype=torch.bfloat16 if out_bf16 else torch.float32, device=X.device)
    st = sb_partial_completion(X, W, M, N, K, lanes, Y, out_bf16, workspace,
                               workspace.numel(), stream)
    if st != SB_OK:
        raise SbError(st, "sb_partial_completion")
    return Y, workspace


def sb_cross_entropy_workspace_bytes(M: int, d: int, V: int) -> int:
    return int(lib().sb_cross_entropy_workspace_bytes(M, d, V))


def sb_cross_entropy_forward(H, W, targets, M, d, V, ignore_index, reduction, z_loss, loss, lse,
                             workspace, workspace_bytes, stream=None) -> int:
    return int(lib().sb_cross_entropy_forward(_ptr(H), _ptr(W), _ptr(targets), M, d, V,
                                              ignore_index, reduction, float(z_loss), _ptr(loss),
                                              _ptr(lse), _ptr(workspace), int(workspace_bytes),
                                              _stream(stream)))


def sb_cross_entropy_backward_workspace_bytes(M: int, d: int, V: int, piece: int, with_dH: bool,
                                              with_dW: bool) -> int:
    return int(lib().sb_cross_entropy_backward_workspace_bytes(M, d, V, piece, int(with_dH),
                                                               int(with_dW)))


def sb_cross_entropy_backward(H, W, targets, lse, grad, M, d, V, ignore_index, reduction, z_loss,
                              piece, dH, dW, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().sb_cross_entropy_backward(_ptr(H), _ptr(W), _ptr(targets), _ptr(lse),
                                               _ptr(grad), M, d, V, ignore_index, reduction,
                                               float(z_loss), piece, _ptr(dH), _ptr(dW),
                                               _ptr(workspace), int(workspace_bytes),
                                               _stream(stream)))


def sb_residual_norm_forward(h, y, pre, post, gate, gate_kind, M, d, stream_type, weight_type,
                             scale, eps, h_out, x, stream=None) -> int:
    return int(lib().sb_residual_norm_forward(_ptr(h), _ptr(y), _ptr(pre), _ptr(post), _ptr(gate),
                                              gate_kind, M, d, stream_type, weight_type,
                                              float(scale), float(eps), _ptr(h_out), _ptr(x),
                                              _stream(stream)))


def sb_residual_norm_workspace_bytes(M: int, d: int) -> int:
    return int(lib().sb_residual_norm_workspace_bytes(M, d))


def sb_residual_norm_backward(dx, dh, h, y, pre, post, gate, gate_kind, M, d, stream_type,
                              weight_type, scale, eps, dh_out, dy, dpre, dpost, dgate, workspace,
                              workspace_bytes, stream=None) -> int:
    return int(lib().sb_residual_norm_backward(
        _ptr(dx), _ptr(dh), _ptr(h), _ptr(y), _ptr(pre), _ptr(post), _ptr(gate), gate_kind, M, d,
        stream_type, weight_type, float(scale), float(eps), _ptr(dh_out), _ptr(dy), _ptr(dpre),
        _ptr(dpost), _ptr(dgate), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def sb_adamw_step(tensors, count, lr, beta1, beta2, eps, step, state_bits, grad_scale=None,
                  stream=None) -> int:
    """tensors: a ctypes array of sb_adamw_tensor (or None for count 0)."""
    return int(lib().sb_adamw_step(tensors, count, lr, beta1, beta2, eps, step, state_bits,
                                   _ptr(grad_scale), _stream(stream)))


def sb_select_source_projection(bytes_ref, bytes_proj, frames_ref, frames_proj,
                                link_bytes_per_s, frame_startup_s, local_proj_s, local_ref_s):
    """Equation (7) plan choice: returns (decision, margin_s); 1 = project at the source."""
    m = ctypes.c_double(0.0)
    d = lib().sb_select_source_projection(float(bytes_ref), float(bytes_proj),
                                          float(frames_ref), float(frames_proj),
                                          float(link_bytes_per_s), float(frame_startup_s),
                                          float(local_proj_s), float(local_ref_s),
                                          ctypes.byref(m))
    return int(d), float(m.value)


def sb_last_device_status(out: sb_outputs) -> int:
    return int(lib().sb_last_device_status(ctypes.byref(out)))


def sb_status_string(status: int) -> str:
    return lib().sb_status_string(status).decode()


def sb_device_info():
    n, cc = ctypes.c_int32(0), ctypes.c_int32(0)
    if lib().sb_device_info(ctypes.byref(n), ctypes.byref(cc)) != 0:
        return None
    return n.value, cc.value


def sb_debug_gumbel_from_bits(bits, g, count: int, stream=None) -> int:
    return int(lib().sb_debug_gumbel_from_bits(_ptr(bits), _ptr(g), int(count), _stream(stream)))


def sb_debug_combine_math(op: int, x, y, count: int, stream=None) -> int:
    return int(lib().sb_debug_combine_math(int(op), _ptr(x), _ptr(y), int(count),
                                           _stream(stream)))


def sb_debug_configure(stall_epilogue: bool, wait_limit_ns: int) -> int:
    return int(lib().sb_debug_configure(1 if stall_epilogue else 0, int(wait_limit_ns)))


def sb_debug_map_encodes() -> int:
    return int(lib().sb_debug_map_encodes())


# ------------------------------------------------------------------ convenience wrapper
def make_outputs(M: int, V: int, k: int, surface: int, *, device="cuda", lse=True,
                 logprob=True, targets=None, workspace=None, topk: int = 0):
    """Allocate the caller-owned buffers of one call with torch; returns (sb_outputs, dict)."""
    import torch
    bufs = {"token": torch.empty(M, dtype=torch.int32, device=device)}
    if logprob or surface in (SB_TOKEN_LOGPROB, SB_GUMBEL_TOKEN):
        bufs["token_logprob"] = torch.empty(M, dtype=torch.float32, device=device)
    if lse:
        bufs["lse"] = torch.empty(M, dtype=torch.float32, device=device)
    if surface == SB_FULL_LOGITS:
        bufs["logits"] = torch.empty(M, V, dtype=torch.bfloat16, device=device)
    if targets is not None:
        bufs["target_ids"] = targets
        bufs["target_logprob"] = torch.empty(M, dtype=torch.float32, device=device)
    if surface == SB_TOPK_LOGPROB:
        bufs["topk_ids"] = torch.empty(M, topk, dtype=torch.int32, device=device)
        bufs["topk_logprob"] = torch.empty(M, topk, dtype=torch.float32, device=device)
    nbytes = sb_workspace_bytes(M, V, k, surface)
    if nbytes == 0:
        raise SbError(SB_ERR_INVALID_ARG, "sb_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    bufs["workspace"] = workspace
    out = sb_outputs(_ptr(bufs["token"]), _ptr(bufs.get("token_logprob")), _ptr(bufs.get("lse")),
                     _ptr(bufs.get("logits")), _ptr(bufs.get("target_ids")),
                     _ptr(bufs.get("target_logprob")), _ptr(workspace),
                     workspace.numel() * workspace.element_size(),
                     _ptr(bufs.get("topk_ids")), _ptr(bufs.get("topk_logprob")), int(topk))
    return out, bufs


class PackedWeights:
    """The packed copy of a [V, d] W for k lane shards (``buf``: a uint8 CUDA tensor), as
    written by ``sb_pack_weights``; pass it as ``W`` to ``project``."""

    def __init__(self, buf, V: int, d: int, k: int):
        self.buf, self.V, self.d, self.k = buf, V, d, k

    def data_ptr(self):
        return self.buf.data_ptr()


def pack_weights(W, k: int, stream=None) -> PackedWeights:
    """Pack the row-major bf16 W [V, d] (CUDA tensor) for k lane shards; enqueued on
    ``stream``."""
    import torch
    V, d = W.shape
    nbytes = sb_packed_weight_bytes(V, d, k)
    if nbytes == 0:
        raise SbError(SB_ERR_INVALID_ARG, "sb_packed_weight_bytes")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    st = sb_pack_weights(W, V, d, k, buf, nbytes, stream)
    if st != SB_OK:
        raise SbError(st, "sb_pack_weights")
    return PackedWeights(buf, V, d, k)


def project(H, W, k: int, surface: int = SB_TOKEN_LOGPROB, *, temperature: float = 1.0,
            seed: int = 0, targets=None, stream=None, lse=True, logprob=True, workspace=None,
            topk: int = 0):
    """Run one projection call on torch CUDA tensors H [M, d] and W [V, d] (bf16), or W a
    ``PackedWeights`` of the same k (then the call reads the packed layout).

    Returns the dict of output tensors (token, token_logprob, lse, logits, target_logprob,
    workspace, as requested). Asynchronous on ``stream``; raises SbError on a bad status."""
    M, d = H.shape
    if isinstance(W, PackedWeights):
        if W.k != k or W.d != d:
            raise SbError(SB_ERR_INVALID_ARG, "project: packed W of another shape")
        V = W.V
        surface |= SB_W_PACKED
    else:
        V = W.shape[0]
    out, bufs = make_outputs(M, V, k, surface & ~SB_W_PACKED, device=H.device, lse=lse,
                             logprob=logprob, targets=targets, workspace=workspace, topk=topk)
    st = sb_lmhead_project(H, W, M, d, V, k, surface, temperature, seed, out, stream)
    if st != SB_OK:
        raise SbError(st, "sb_lmhead_project")
    bufs["_outputs"] = out
    return bufs


# ------------------------------------------------------------------ training the head
def _tensor(name, t, shape, dtypes, device, where):
    """Refuses a tensor the kernels would misread: another shape or type, one that is not
    contiguous, or one that is not on the current CUDA device (its index: `device`)."""
    if (t.shape == shape and t.dtype in dtypes and t.get_device() == device and
            t.is_contiguous()):
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{where}: {name} is {t.dtype}, not {' or '.join(map(str, dtypes))}")
    if t.get_device() != device:
        raise ValueError(f"{where}: {name} is on {t.device}, not cuda:{device}")
    raise ValueError(f"{where}: {name} is not contiguous")


def _current(device):
    """The raw handle of torch's current stream (a tenth of current_stream()'s time)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device)


def _on_stream(stream, call, *tensors):
    """call() with `stream` (a torch stream or a raw handle) as torch's current one, so that what
    it allocates belongs to the stream its kernels run on; torch's allocator learns that the
    given tensors (None are skipped) are read there, and keeps their memory until then."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    with torch.cuda.stream(stream):
        out = call()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return out


def _reduction(reduction, where):
    try:
        return REDUCTIONS[reduction]
    except KeyError:
        raise ValueError(f"{where}: reduction is one of {sorted(REDUCTIONS)}, "
                         f"not {reduction!r}") from None


def _loss_problem(H, W, targets, ignore_index, where):
    """Checks the arguments both directions share; returns (M, d, V, device index)."""
    import torch
    if not -2 ** 31 <= ignore_index < 2 ** 31:  # the C call would take its lowest 32 bits
        raise ValueError(f"{where}: ignore_index {ignore_index} is not a 32-bit integer")
    dev = torch.cuda.current_device()
    if H.dim() != 2 or W.dim() != 2:
        raise ValueError(f"{where}: H is [M, d] and W [V, d]")
    M, d = H.shape
    V, dw = W.shape
    bf16 = torch.bfloat16
    if not (dw == d and H.dtype is bf16 and W.dtype is bf16 and targets.dtype is torch.int32 and
            targets.shape == (M,) and H.get_device() == dev and W.get_device() == dev and
            targets.get_device() == dev and H.is_contiguous() and W.is_contiguous() and
            targets.is_contiguous()):
        _tensor("H", H, (M, d), (bf16,), dev, where)
        _tensor("W", W, (V, d), (bf16,), dev, where)
        _tensor("targets", targets, (M,), (torch.int32,), dev, where)
    return M, d, V, dev


def _workspace(workspace, device, where):
    """Refuses a workspace that the kernels cannot write to; returns its size in bytes."""
    if workspace.get_device() != device:
        raise ValueError(f"{where}: workspace is on {workspace.device}, not cuda:{device}")
    if not workspace.is_contiguous():
        raise ValueError(f"{where}: workspace is not contiguous")
    return workspace.nbytes


def _nonzero(nbytes, where):
    if nbytes == 0:
        raise SbError(SB_ERR_INVALID_ARG, where)
    return nbytes


def cross_entropy(H, W, targets, *, ignore_index: int = -100, z_loss: float = 0.0,
                  reduction: str = "mean", stream=None, workspace=None):
    """The cross entropy of the rows' targets under logits H Wᵀ, without keeping the logits:
    lse - z_target + z_loss lse² per row, 0 for rows whose target is ``ignore_index``.

    H [M, d] and W [V, d] bf16, targets [M] int32, contiguous CUDA tensors. Returns a dict:
    loss (float32, [M] for reduction "none", [1] for "sum" and "mean"), lse [M] and workspace.
    Asynchronous on ``stream``; raises SbError on a bad status. A target outside [0, V) that is
    not ``ignore_index`` gives a NaN loss, and ``device_status`` of the workspace reports it. No
    autograd graph is built, whatever the inputs ask for: ``cross_entropy_backward`` gives the
    gradients (int64 labels are converted by ``targets.int()``)."""
    if stream is not None:
        return _on_stream(stream, lambda: cross_entropy(
            H, W, targets, ignore_index=ignore_index, z_loss=z_loss, reduction=reduction,
            workspace=workspace), H, W, targets, workspace)
    import torch
    red = _reduction(reduction, "cross_entropy")
    M, d, V, dev = _loss_problem(H, W, targets, ignore_index, "cross_entropy")
    L = lib()
    if workspace is None:
        size = _nonzero(L.sb_cross_entropy_workspace_bytes(M, d, V), "cross_entropy")
        workspace = torch.empty(size, dtype=torch.uint8, device=H.device)
    else:
        size = _workspace(workspace, dev, "cross_entropy")
    loss = torch.empty(M if red == SB_REDUCE_NONE else 1, dtype=torch.float32, device=H.device)
    lse = torch.empty(M, dtype=torch.float32, device=H.device)
    st = L.sb_cross_entropy_forward(H.data_ptr(), W.data_ptr(), targets.data_ptr(), M, d, V,
                                    ignore_index, red, z_loss, loss.data_ptr(), lse.data_ptr(),
                                    workspace.data_ptr(), size, _current(dev))
    if st != SB_OK:
        raise SbError(st, "sb_cross_entropy_forward")
    return {"loss": loss, "lse": lse, "workspace": workspace}


def cross_entropy_backward(H, W, targets, lse, *, grad=None, ignore_index: int = -100,
                           z_loss: float = 0.0, reduction: str = "mean", need_dH: bool = True,
                           need_dW: bool = True, piece: int = 0, stream=None, workspace=None):
    """The gradients of ``cross_entropy`` in H and W, bf16, from its ``lse`` and the same
    arguments; ``grad`` is the incoming gradient (float32, [M] for "none", else [1]; None stands
    for ones). The vocabulary is worked off in pieces of ``piece`` columns (0: the library's
    choice). Returns a dict: dH, dW (None where not needed) and workspace."""
    if stream is not None:
        return _on_stream(stream, lambda: cross_entropy_backward(
            H, W, targets, lse, grad=grad, ignore_index=ignore_index, z_loss=z_loss,
            reduction=reduction, need_dH=need_dH, need_dW=need_dW, piece=piece,
            workspace=workspace), H, W, targets, lse, grad, workspace)
    import torch
    where = "cross_entropy_backward"
    red = _reduction(reduction, where)
    M, d, V, dev = _loss_problem(H, W, targets, ignore_index, where)
    _tensor("lse", lse, (M,), (torch.float32,), dev, where)
    if grad is not None:
        _tensor("grad", grad, (M if red == SB_REDUCE_NONE else 1,), (torch.float32,), dev, where)
    L = lib()
    if workspace is None:
        size = _nonzero(
            L.sb_cross_entropy_backward_workspace_bytes(M, d, V, piece, need_dH, need_dW), where)
        workspace = torch.empty(size, dtype=torch.uint8, device=H.device)
    else:
        size = _workspace(workspace, dev, where)
    dH = torch.empty_like(H) if need_dH else None
    dW = torch.empty_like(W) if need_dW else None
    st = L.sb_cross_entropy_backward(H.data_ptr(), W.data_ptr(), targets.data_ptr(),
                                     lse.data_ptr(), _ptr(grad), M, d, V, ignore_index, red,
                                     z_loss, piece, _ptr(dH), _ptr(dW), workspace.data_ptr(),
                                     size, _current(dev))
    if st != SB_OK:
        raise SbError(st, "sb_cross_entropy_backward")
    return {"dH": dH, "dW": dW, "workspace": workspace}


def device_status(workspace) -> int:
    """``sb_last_device_status`` of a workspace tensor (synchronises)."""
    return sb_last_device_status(sb_outputs(workspace=_ptr(workspace),
                                            workspace_bytes=workspace.nbytes))


def _norm_problem(h, y, pre, post, gate, where):
    """Checks the arguments both directions share; returns (M, d, gate kind, the types of the
    stream and of the weights, device index)."""
    import torch
    dev = torch.cuda.current_device()
    if h.dim() != 2:
        raise ValueError(f"{where}: h is [M, d]")
    M, d = h.shape
    f32, bf16 = torch.float32, torch.bfloat16
    ht, wt = h.dtype, pre.dtype
    kind = SB_GATE_NONE
    if gate is not None:
        kind = SB_GATE_CHANNEL if gate.dim() == 1 else SB_GATE_TOKEN
    gs, gt = ((d,), wt) if kind == SB_GATE_CHANNEL else ((M, d), bf16)
    if not ((ht is bf16 or ht is f32) and (wt is bf16 or wt is f32) and y.dtype is bf16 and
            y.shape == (M, d) and pre.shape == (d,) and h.get_device() == dev and
            y.get_device() == dev and pre.get_device() == dev and h.is_contiguous() and
            y.is_contiguous() and pre.is_contiguous()):
        _tensor("h", h, (M, d), (bf16, f32), dev, where)
        _tensor("y", y, (M, d), (bf16,), dev, where)
        _tensor("pre", pre, (d,), (bf16, f32), dev, where)
    if post is not None:
        _tensor("post", post, (d,), (wt,), dev, where)
    if gate is not None:
        _tensor("gate", gate, gs, (gt,), dev, where)
    return (M, d, kind, SB_F32 if ht is f32 else SB_BF16, SB_F32 if wt is f32 else SB_BF16, dev)


def residual_norm(h, y, pre, *, post=None, gate=None, scale: float = 1.0, eps: float = 1e-6,
                  stream=None):
    """The end of a block: h' = scale h + gate n(y; post) and x = n(h'; pre), with
    n(x; w) = w x / sqrt(mean(x²) + eps) over the last axis.

    h [M, d] bf16 or float32 (the residual stream), y [M, d] bf16 (the block's output), pre and
    post [d] of one type, bf16 or float32 (post None: no norm of y), gate [d] of that type,
    [M, d] bf16, or None. Returns a dict: h (h', of h's type) and x (bf16: what the next block,
    or ``project`` and ``cross_entropy``, read). Asynchronous on ``stream``. No autograd graph is
    built: ``residual_norm_backward`` gives the gradients."""
    if stream is not None:
        return _on_stream(stream, lambda: residual_norm(
            h, y, pre, post=post, gate=gate, scale=scale, eps=eps), h, y, pre, post, gate)
    import torch
    M, d, kind, ht, wt, dev = _norm_problem(h, y, pre, post, gate, "residual_norm")
    h_out, x = torch.empty_like(h), torch.empty_like(y)
    st = lib().sb_residual_norm_forward(h.data_ptr(), y.data_ptr(), pre.data_ptr(), _ptr(post),
                                        _ptr(gate), kind, M, d, ht, wt, scale, eps,
                                        h_out.data_ptr(), x.data_ptr(), _current(dev))
    if st != SB_OK:
        raise SbError(st, "sb_residual_norm_forward")
    return {"h": h_out, "x": x}


def residual_norm_backward(dx, dh, h, y, pre, *, post=None, gate=None, scale: float = 1.0,
                           eps: float = 1e-6, stream=None, workspace=None):
    """The gradients of ``residual_norm``: dx [M, d] bf16 is the gradient of its x, dh that of
    its h' (None: nothing else reads h'), ``h`` the h' that it returned; the rest as there.
    Returns a dict: dh (the gradient of the incoming stream), dy, dpre, dpost, dgate (None where
    there is no such input) and workspace. The weights' gradients have the weights' type."""
    if stream is not None:
        return _on_stream(stream, lambda: residual_norm_backward(
            dx, dh, h, y, pre, post=post, gate=gate, scale=scale, eps=eps, workspace=workspace),
            dx, dh, h, y, pre, post, gate, workspace)
    import torch
    where = "residual_norm_backward"
    M, d, kind, ht, wt, dev = _norm_problem(h, y, pre, post, gate, where)
    _tensor("dx", dx, (M, d), (torch.bfloat16,), dev, where)
    if dh is not None:
        _tensor("dh", dh, (M, d), (h.dtype,), dev, where)
    L = lib()
    if workspace is None:
        size = _nonzero(L.sb_residual_norm_workspace_bytes(M, d), where)
        workspace = torch.empty(size, dtype=torch.uint8, device=h.device)
    else:
        size = _workspace(workspace, dev, where)
    dh_out, dy, dpre = torch.empty_like(h), torch.empty_like(y), torch.empty_like(pre)
    dpost = None if post is None else torch.empty_like(post)
    dgate = None if gate is None else torch.empty_like(gate)
    st = L.sb_residual_norm_backward(dx.data_ptr(), _ptr(dh), h.data_ptr(), y.data_ptr(),
                                     pre.data_ptr(), _ptr(post), _ptr(gate), kind, M, d, ht, wt,
                                     scale, eps, dh_out.data_ptr(), dy.data_ptr(),
                                     dpre.data_ptr(), _ptr(dpost), _ptr(dgate),
                                     workspace.data_ptr(), size, _current(dev))
    if st != SB_OK:
        raise SbError(st, "sb_residual_norm_backward")
    return {"dh": dh_out, "dy": dy, "dpre": dpre, "dpost": dpost, "dgate": dgate,
            "workspace": workspace}


class AdamW:
    """AdamW over a list of tensors, updated in place by one kernel launch per step
    (``sb_adamw_step``; its formulas and formats are described in sb.h).

    params: contiguous CUDA tensors, bf16 or float32, of any shape. grads: one for each, of the
    same shape, bf16 or float32; they are read by every ``step`` (give new ones to ``step`` when
    they move). masters: float32 copies of bf16 parameters (a list with None where a parameter
    has none, or None for none at all). state_bits: 32, or 8 for E4M3 codes in blocks of 256
    values. states: existing moments, a tuple for each parameter, ``(m, v)`` float32 or
    ``(m, root, m_scale, root_scale)`` with float8_e4m3fn codes; None starts from zeros.
    weight_decay: one number, or one for each parameter. step: steps already taken.

    The handle keeps the tensors' addresses (and their memory): a parameter, copy or state that is
    given other memory later (``x.data = ...``) needs a new handle. In a CUDA graph a step is
    captured with its rate and step number, so that every replay repeats that step's bias
    correction: capture the forward and backward calls and step outside, or capture per step."""

    def __init__(self, params, grads=None, *, lr: float = 1e-3, betas=(0.9, 0.999),
                 eps: float = 1e-8, weight_decay=0.01, state_bits: int = 32, masters=None,
                 states=None, step: int = 0):
        import torch
        where = "AdamW"
        if state_bits not in (8, 32):
            raise ValueError(f"{where}: state_bits is 8 or 32, not {state_bits!r}")
        self.params = list(params)
        n = len(self.params)
        self.lr, self.betas, self.eps = lr, tuple(betas), eps
        self.state_bits, self.step_count = state_bits, step
        self.masters = [None] * n if masters is None else list(masters)
        decay = (list(weight_decay) if isinstance(weight_decay, (list, tuple))
                 else [weight_decay] * n)
        self.states = [None] * n if states is None else [tuple(s) for s in states]
        for name, x in (("masters", self.masters), ("weight_decay", decay),
                        ("states", self.states)):
            if len(x) != n:
                raise ValueError(f"{where}: {len(x)} {name} for {n} parameters")
        self._device = torch.cuda.current_device()
        dev, bf16, f32 = self._device, torch.bfloat16, torch.float32
        code = torch.float8_e4m3fn if state_bits == 8 else f32
        self._list = (sb_adamw_tensor * n)()
        written = []  # (first byte, byte past the end) of every array that a step writes
        for i, (p, w, t) in enumerate(zip(self.params, self.masters, self._list)):
            _tensor(f"params[{i}]", p, p.shape, (bf16, f32), dev, where)
            k = p.numel()
            if w is not None:
                if p.dtype is not bf16:
                    raise TypeError(f"{where}: params[{i}] is float32 and has no master")
                _tensor(f"masters[{i}]", w, p.shape, (f32,), dev, where)
                t.master = w.data_ptr()
            shapes = ((k, code), (k, code))
            if state_bits == 8:
                shapes += (((k + 255) // 256, f32),) * 2
            s = self.states[i]
            if s is None:
                s = self.states[i] = tuple(p.new_zeros(c, dtype=d) for c, d in shapes)
            if len(s) != len(shapes):
                raise ValueError(f"{where}: states[{i}] has {len(s)} tensors, not {len(shapes)}")
            for j, (x, (c, d)) in enumerate(zip(s, shapes)):
                if x.numel() != c:
                    raise ValueError(f"{where}: states[{i}][{j}] has {x.numel()} values, not {c}")
                _tensor(f"states[{i}][{j}]", x, x.shape, (d,), dev, where)
            t.param, t.exp_avg, t.exp_avg_sq = p.data_ptr(), s[0].data_ptr(), s[1].data_ptr()
            if state_bits == 8:
                t.scale, t.scale_sq = s[2].data_ptr(), s[3].data_ptr()
            written += [(x.data_ptr(), x.data_ptr() + x.nbytes)
                        for x in (p, w, *s) if x is not None and k]
            t.n, t.weight_decay = k, decay[i]
            t.param_type = SB_F32 if p.dtype is f32 else SB_BF16
        written.sort()
        if any(a[1] > b[0] for a, b in zip(written, written[1:])):
            raise ValueError(f"{where}: tensors overlap (two blocks of a launch would write them)")
        # the descriptors hold addresses: these keep the memory there, whatever becomes of the tensors
        self._memory = [x.untyped_storage() for q in (self.params, self.masters, *self.states)
                        for x in q if x is not None]
        self._streams = set()
        self.grads = None
        if grads is not None:
            self._bind(grads)

    def _bind(self, grads):
        import torch
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"AdamW: {len(grads)} gradients for {len(self.params)} parameters")
        # every check before the first address: a refused list leaves the bound one as it was
        dev, types = self._device, (torch.bfloat16, torch.float32)
        for i, (g, p) in enumerate(zip(grads, self.params)):
            if not (g.shape == p.shape and g.dtype in types and g.get_device() == dev and
                    g.is_contiguous()):
                _tensor(f"grads[{i}]", g, p.shape, types, dev, "AdamW")
        for g, t in zip(grads, self._list):
            t.grad = g.data_ptr()
            t.grad_type = SB_F32 if g.dtype == torch.float32 else SB_BF16
        self.grads = grads
        self._grad_memory = [g.untyped_storage() for g in grads]

    def step(self, grads=None, *, grad_scale=None, lr=None, stream=None) -> None:
        """One step, asynchronous on ``stream``: ``grads`` replaces the gradients bound so far,
        ``grad_scale`` (float32 [1] on the device) multiplies them, ``lr`` replaces the rate."""
        import torch
        # the launch goes to the current device, the addresses are those of the handle's
        device = torch.cuda.current_device()
        if stream is not None and device == self._device:
            device = getattr(stream, "device_index", device)
        if device != self._device:
            raise ValueError(f"AdamW: the tensors are on cuda:{self._device}, the step would run "
                             f"on device {device}")
        on = _current(device) if stream is None else stream
        if grad_scale is not None:
            _tensor("grad_scale", grad_scale, (1,), (torch.float32,), self._device, "AdamW")
        if grads is not None:
            self._bind(grads)
        if self.grads is None and self.params:
            raise ValueError("AdamW: no gradients have been given")
        rate = self.lr if lr is None else lr
        st = sb_adamw_step(self._list, len(self.params), rate, self.betas[0], self.betas[1],
                           self.eps, self.step_count + 1, self.state_bits, grad_scale, on)
        if st != SB_OK:
            raise SbError(st, "sb_adamw_step")
        self.lr = rate
        self.step_count += 1
        if stream is not None:  # any of these may be let go of while that stream uses them
            own = ()
            if _stream(stream) not in self._streams:  # once is enough for what stays bound
                self._streams.add(_stream(stream))
                own = (*self.params, *self.masters, *(x for s in self.states for x in s))
            _on_stream(stream, lambda: None, grad_scale, *(self.grads or ()), *own)
