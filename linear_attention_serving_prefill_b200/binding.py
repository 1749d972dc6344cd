"""Thin ctypes binding of libkda_b200.so (argument marshalling only).

Every function here checks tensor placement and dtype, passes raw device
pointers and sizes to the C ABI declared in ``include/kda.h``, and raises
``KdaError`` on a non-zero status.  All arithmetic runs in the CUDA library;
there is no fallback: if the library is missing the import of this module
fails.  Outputs and workspaces that a call makes belong to its ``stream``, as
tensors made under ``torch.cuda.stream(stream)`` do.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libkda_b200.so")

KDA_DTYPE = {torch.bfloat16: 0, torch.float32: 1}
KDA_ALGO = {"auto": 0, "cuda_core": 1, "tensor_core": 2, "tensor_core_split": 3}
KDA_GATE = {"bounded": 0, "softplus": 1}
STATUS_NAMES = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED",
                3: "KDA_ERR_WORKSPACE", 4: "KDA_ERR_CUDA", 5: "KDA_ERR_TIMEOUT"}

# Every exported symbol of include/kda.h, with its ctypes signature.
_P, _I32, _SZ, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "kda_abi_version": ([], _I32),
    "kda_status_string": ([_I32], ctypes.c_char_p),
    "kda_prefill_workspace_size": ([_I32, _I32, _I32, _I32, _I32, _I32, _I32], _SZ),
    "kda_prefill_gated_workspace_size": ([_I32] * 8, _SZ),
    "kda_prefill": ([_P] * 8 + [_I32] * 6 + [_P] * 4 + [_SZ, _P], _I32),
    "kda_prefill_ex": ([_P] * 8 + [_I32] * 6 + [_P] * 4 + [_SZ, _I32, _P, _P, _I32], _I32),
    "kda_prefill_kernel_count": ([_I32] * 7, _I32),
    "kda_prefill_segments": ([_I32] * 7, _I32),
    "kda_prefill_checkpointed": ([_P] * 8 + [_I32] * 6 + [_P] * 4 + [_SZ, _I32, _P, _P, _I32, _I32, _P],
                                 _I32),
    "kda_checkpoint_count": ([_P, _I32, _I32], ctypes.c_int64),
    "kda_prefill_noalloc": ([_P] * 8 + [_I32] * 6 + [_P] * 4, _I32),
    "kda_decode_step": ([_P] * 6 + [_I32] * 5 + [_P, _I32, _P, _P, _P], _I32),
    "kda_decode_step_gated": ([_P] * 6 + [_I32] * 5 + [_P, _I32, _P, _P, _I32, _P], _I32),
    "kda_prefill_gated": ([_P] * 8 + [_I32] * 6 + [_P] * 4 + [_SZ, _I32, _I32, _P], _I32),
    "kda_prefill_debug": ([_P] * 8 + [_I32] * 6 + [_P] * 4 + [_SZ] + [_P] * 5, _I32),
    "kda_decode_check_slots": ([_P, _I32, _I32], _I32),
    "kda_device_status": ([_P, _P], _I32),
    "kda_decode_multi": ([_P] * 6 + [_I32] * 6 + [_P, _I32, _P, _P, _I32, _P, _P], _I32),
    "kda_selftest_wait_timeout": ([ctypes.c_int64, _P], _I32),
    "kda_gdr_prefill_workspace_size": ([_I32] * 8, _SZ),
    "kda_gdr_prefill": ([_P] * 7 + [_I32] * 7 + [_F32, _P, _I32] + [_P] * 4 + [_I32] * 2
                        + [_P] * 2 + [_SZ, _I32, _P], _I32),
    "kda_gdr_decode": ([_P] * 5 + [_I32] * 7 + [_F32, _P, _I32] + [_P] * 3 + [_I32] + [_P] * 2,
                       _I32),
    "kda_gdr_decode_blocks": ([_P] * 5 + [_I32] * 7 + [_F32, _P, _I32] + [_P] * 5 + [_I32] * 2
                              + [_P] * 2, _I32),
    "kda_block_plan": ([_P] * 2 + [_I32, _P, _I32, _P, _P] + [_I32] * 3 + [_P] * 7, _I32),
}


class KdaError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} "
                         f"({_lib.kda_status_string(code).decode()})")
        self.code = code


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"KDA CUDA library not built: {_LIB_PATH} is missing "
                          "(run python -m linear_attention_serving_prefill_b200.build)")
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    return lib


_lib = _load()


def library_path() -> str:
    return _LIB_PATH


def kda_status_string(code: int) -> str:
    return _lib.kda_status_string(code).decode()


def _check(code: int, where: str):
    if code != 0:
        raise KdaError(code, where)


def _dev(t: Optional[torch.Tensor], name: str, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _made(stream, make, *args, **kw):
    """make(*args, **kw), its memory belonging to ``stream`` (None: the current one).  Kernels on
    another stream than a tensor's own would write while the allocator's earlier or later
    tenants of that memory are in use."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _stream_ptr(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def kda_prefill_workspace_size(total_tokens: int, num_seqs: int, H: int, dk: int, dv: int,
                               dtype=torch.bfloat16, algo: str = "auto") -> int:
    return int(_lib.kda_prefill_workspace_size(total_tokens, num_seqs, H, dk, dv,
                                               KDA_DTYPE[dtype], KDA_ALGO[algo]))


def kda_prefill_gated_workspace_size(total_tokens: int, num_seqs: int, H: int, dk: int, dv: int,
                                     dtype=torch.bfloat16, algo: str = "auto",
                                     gate: str = "bounded") -> int:
    return int(_lib.kda_prefill_gated_workspace_size(total_tokens, num_seqs, H, dk, dv,
                                                     KDA_DTYPE[dtype], KDA_ALGO[algo],
                                                     KDA_GATE[gate]))


def kda_prefill(q, k, v, z, A, beta, cu_seqlens, cu_seqlens_host=None, initial_state=None,
                output_final_state: bool = True, final_state=None, o=None, workspace=None,
                algo: str = "auto", stream=None, stage_events=None, gate: str = "bounded"):
    """Chunked KDA prefill over packed sequences; returns ``(o, final_state)``.

    q, k, z [T,H,dk], v [T,H,dv] (bf16 or fp32, one dtype); A [H,dk] fp32;
    beta [T,H] fp32; cu_seqlens [N+1] int32 on the device; cu_seqlens_host an
    optional CPU copy; initial_state [N,H,dk,dv] fp32 or None.  ``final_state``
    may be passed (e.g. ``initial_state`` itself, for in-place resume);
    otherwise it is allocated when ``output_final_state``.  ``stage_events``
    (a list of recorded ``torch.cuda.Event``) receives the kernel boundaries.
    ``gate="softplus"`` selects the unbounded gate (kda_prefill_gated; no events).
    """
    T, H, dk = q.shape
    dv = v.shape[2]
    N = cu_seqlens.shape[0] - 1
    dt = q.dtype
    if dt not in KDA_DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    if o is None:
        o = _made(stream, torch.empty, T, H, dv, dtype=dt, device=q.device)
    if final_state is None and output_final_state:
        final_state = _made(stream, torch.empty, N, H, dk, dv, dtype=torch.float32, device=q.device)
    need = kda_prefill_gated_workspace_size(T, N, H, dk, dv, dt, algo, gate)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = _made(stream, torch.empty, need, dtype=torch.uint8, device=q.device)
    host = None
    if cu_seqlens_host is not None:
        ch = cu_seqlens_host.to(torch.int32).contiguous()
        host = ctypes.c_void_p(ch.data_ptr())
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if gate != "bounded":
        if stage_events:
            raise ValueError("stage events are recorded for the lower-bounded gate only")
        code = _lib.kda_prefill_gated(
            _dev(q, "q", dt), _dev(k, "k", dt), _dev(v, "v", dt), _dev(z, "z", dt),
            _dev(A, "A", torch.float32), _dev(beta, "beta", torch.float32),
            _dev(cu_seqlens, "cu_seqlens", torch.int32), host, N, T, H, dk, dv, KDA_DTYPE[dt],
            _dev(initial_state, "initial_state", torch.float32),
            _dev(final_state, "final_state", torch.float32), _dev(o, "o", dt),
            _dev(workspace, "workspace"), ws_bytes, KDA_ALGO[algo], KDA_GATE[gate],
            _stream_ptr(stream))
        _check(code, "kda_prefill_gated")
        return o, final_state
    ev_arr, n_ev = None, 0
    if stage_events:
        ev_arr = (ctypes.c_void_p * len(stage_events))(*[e.cuda_event for e in stage_events])
        n_ev = len(stage_events)
    code = _lib.kda_prefill_ex(
        _dev(q, "q", dt), _dev(k, "k", dt), _dev(v, "v", dt), _dev(z, "z", dt),
        _dev(A, "A", torch.float32), _dev(beta, "beta", torch.float32),
        _dev(cu_seqlens, "cu_seqlens", torch.int32), host, N, T, H, dk, dv, KDA_DTYPE[dt],
        _dev(initial_state, "initial_state", torch.float32),
        _dev(final_state, "final_state", torch.float32), _dev(o, "o", dt),
        _dev(workspace, "workspace"), ws_bytes, KDA_ALGO[algo], _stream_ptr(stream), ev_arr, n_ev)
    _check(code, "kda_prefill")
    return o, final_state


def kda_checkpoint_count(cu_seqlens_host, checkpoint_every: int) -> int:
    """Rows of the checkpoint tensor: sum over sequences of L_n // checkpoint_every."""
    ch = cu_seqlens_host.to(torch.int32).contiguous()
    n = _lib.kda_checkpoint_count(ctypes.c_void_p(ch.data_ptr()), ch.numel() - 1, checkpoint_every)
    if n < 0:
        raise KdaError(1, "kda_checkpoint_count")
    return int(n)


def kda_prefill_checkpointed(q, k, v, z, A, beta, cu_seqlens, cu_seqlens_host, checkpoint_every,
                             initial_state=None, final_state=None, o=None, checkpoints=None,
                             workspace=None, algo: str = "auto", stream=None):
    """kda_prefill plus the state after every ``checkpoint_every`` tokens of each
    sequence; returns ``(o, final_state, checkpoints [count, H, dk, dv])``."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = cu_seqlens.shape[0] - 1
    dt = q.dtype
    if o is None:
        o = _made(stream, torch.empty, T, H, dv, dtype=dt, device=q.device)
    if final_state is None:
        final_state = _made(stream, torch.empty, N, H, dk, dv, dtype=torch.float32, device=q.device)
    count = kda_checkpoint_count(cu_seqlens_host, checkpoint_every)
    if checkpoints is None:
        checkpoints = _made(stream, torch.empty, max(count, 1), H, dk, dv, dtype=torch.float32,
                            device=q.device)
    need = kda_prefill_workspace_size(T, N, H, dk, dv, dt, algo)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = _made(stream, torch.empty, need, dtype=torch.uint8, device=q.device)
    ch = cu_seqlens_host.to(torch.int32).contiguous()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = _lib.kda_prefill_checkpointed(
        _dev(q, "q", dt), _dev(k, "k", dt), _dev(v, "v", dt), _dev(z, "z", dt),
        _dev(A, "A", torch.float32), _dev(beta, "beta", torch.float32),
        _dev(cu_seqlens, "cu_seqlens", torch.int32), ctypes.c_void_p(ch.data_ptr()), N, T, H, dk,
        dv, KDA_DTYPE[dt], _dev(initial_state, "initial_state", torch.float32),
        _dev(final_state, "final_state", torch.float32), _dev(o, "o", dt),
        _dev(workspace, "workspace"), ws_bytes, KDA_ALGO[algo], _stream_ptr(stream), None, 0,
        int(checkpoint_every), _dev(checkpoints, "checkpoints", torch.float32))
    _check(code, "kda_prefill_checkpointed")
    return o, final_state, checkpoints[:count]


def kda_prefill_noalloc(q, k, v, z, A, beta, cu_seqlens, cu_seqlens_host=None,
                        initial_state=None, output_final_state: bool = True, final_state=None,
                        o=None, stream=None):
    """kda_prefill with the library's fixed scratch array instead of a workspace.

    For callers that must not allocate device memory during the call: pass
    preallocated ``o`` (and ``final_state``) to keep this function from
    allocating them.  Returns ``(o, final_state)``.
    """
    T, H, dk = q.shape
    dv = v.shape[2]
    N = cu_seqlens.shape[0] - 1
    dt = q.dtype
    if dt not in KDA_DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    if o is None:
        o = _made(stream, torch.empty, T, H, dv, dtype=dt, device=q.device)
    if final_state is None and output_final_state:
        final_state = _made(stream, torch.empty, N, H, dk, dv, dtype=torch.float32, device=q.device)
    host = None
    if cu_seqlens_host is not None:
        ch = cu_seqlens_host.to(torch.int32).contiguous()
        host = ctypes.c_void_p(ch.data_ptr())
    code = _lib.kda_prefill_noalloc(
        _dev(q, "q", dt), _dev(k, "k", dt), _dev(v, "v", dt), _dev(z, "z", dt),
        _dev(A, "A", torch.float32), _dev(beta, "beta", torch.float32),
        _dev(cu_seqlens, "cu_seqlens", torch.int32), host, N, T, H, dk, dv, KDA_DTYPE[dt],
        _dev(initial_state, "initial_state", torch.float32),
        _dev(final_state, "final_state", torch.float32), _dev(o, "o", dt), _stream_ptr(stream))
    _check(code, "kda_prefill_noalloc")
    return o, final_state


def kda_prefill_kernel_count(T: int, N: int, H: int, dk: int, dv: int, dtype=torch.bfloat16,
                             algo: str = "auto") -> int:
    return int(_lib.kda_prefill_kernel_count(T, N, H, dk, dv, KDA_DTYPE[dtype], KDA_ALGO[algo]))


def kda_prefill_segments(T: int, N: int, H: int, dk: int, dv: int, dtype=torch.bfloat16,
                         algo: str = "auto") -> int:
    """Segments per sequence the call uses (1 = no split, 0 = invalid arguments)."""
    return int(_lib.kda_prefill_segments(T, N, H, dk, dv, KDA_DTYPE[dtype], KDA_ALGO[algo]))


def kda_decode_step(q, k, v, z, A, beta, state, slots=None, o=None, stream=None,
                    gate: str = "bounded"):
    """One decode step; ``state`` [P,H,dk,dv] fp32 is updated in place; returns o."""
    B, H, dk = q.shape
    dv = v.shape[2]
    dt = q.dtype
    if o is None:
        o = _made(stream, torch.empty, B, H, dv, dtype=dt, device=q.device)
    code = _lib.kda_decode_step_gated(
        _dev(q, "q", dt), _dev(k, "k", dt), _dev(v, "v", dt), _dev(z, "z", dt),
        _dev(A, "A", torch.float32), _dev(beta, "beta", torch.float32), B, H, dk, dv,
        KDA_DTYPE[dt], _dev(state, "state", torch.float32), state.shape[0],
        _dev(slots, "slots", torch.int32), _dev(o, "o", dt), KDA_GATE[gate], _stream_ptr(stream))
    _check(code, "kda_decode_step")
    return o


def kda_decode_multi(q, k, v, z, A, beta, state, slots=None, num_tokens=None,
                     update_state: bool = False, o=None, want_outputs: bool = True, stream=None):
    """Speculative-decoding verify (update_state=False: outputs for every draft
    token, state untouched) or replay (update_state=True: advance each sequence's
    state by its first num_tokens[b] tokens in place).

    q, k, z [B,Tq,H,dk], v [B,Tq,H,dv]; beta [B,Tq,H] fp32; state [P,H,dk,dv] fp32.
    Returns o [B,Tq,H,dv] (or None when want_outputs is False in replay mode).
    """
    B, Tq, H, dk = q.shape
    dv = v.shape[3]
    dt = q.dtype
    if o is None and (want_outputs or not update_state):
        o = _made(stream, torch.empty, B, Tq, H, dv, dtype=dt, device=q.device)
    code = _lib.kda_decode_multi(
        _dev(q, "q", dt), _dev(k, "k", dt), _dev(v, "v", dt), _dev(z, "z", dt),
        _dev(A, "A", torch.float32), _dev(beta, "beta", torch.float32), B, Tq, H, dk, dv,
        KDA_DTYPE[dt], _dev(state, "state", torch.float32), state.shape[0],
        _dev(slots, "slots", torch.int32), _dev(num_tokens, "num_tokens", torch.int32),
        1 if update_state else 0, _dev(o, "o", dt), _stream_ptr(stream))
    _check(code, "kda_decode_multi")
    return o


def kda_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Enqueue the bounded-wait self-test; read the result with kda_device_status()."""
    _check(_lib.kda_selftest_wait_timeout(int(limit_ns), _stream_ptr(stream)),
           "kda_selftest_wait_timeout")


def kda_device_status(stream=None) -> int:
    out = ctypes.c_int32(0)
    _check(_lib.kda_device_status(_stream_ptr(stream), ctypes.byref(out)), "kda_device_status")
    return int(out.value)


def kda_prefill_debug(q, k, v, z, A, beta, cu_seqlens, cu_seqlens_host, initial_state=None,
                      stream=None):
    """Tensor-core prefill plus its stage intermediates; returns a dict with o,
    final_state and G, W, U, delta (fp32 [T, H, 128], see include/kda.h)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = cu_seqlens.shape[0] - 1
    dt = q.dtype
    dev = q.device
    out = {"o": _made(stream, torch.empty, T, H, dv, dtype=dt, device=dev),
           "final_state": _made(stream, torch.empty, N, H, dk, dv, dtype=torch.float32, device=dev)}
    for name, d in (("G", dk), ("W", dk), ("U", dv), ("delta", dv)):
        out[name] = _made(stream, torch.full, (T, H, d), float("nan"), dtype=torch.float32, device=dev)
    need = kda_prefill_workspace_size(T, N, H, dk, dv, dt, "tensor_core")
    ws = _made(stream, torch.empty, max(need, 1), dtype=torch.uint8, device=dev)
    ch = cu_seqlens_host.to(torch.int32).contiguous()
    code = _lib.kda_prefill_debug(
        _dev(q, "q", dt), _dev(k, "k", dt), _dev(v, "v", dt), _dev(z, "z", dt),
        _dev(A, "A", torch.float32), _dev(beta, "beta", torch.float32),
        _dev(cu_seqlens, "cu_seqlens", torch.int32), ctypes.c_void_p(ch.data_ptr()), N, T, H, dk,
        dv, KDA_DTYPE[dt], _dev(initial_state, "initial_state", torch.float32),
        _dev(out["final_state"], "final_state", torch.float32), _dev(out["o"], "o", dt),
        _dev(ws, "workspace"), need, _dev(out["G"], "G"), _dev(out["W"], "W"), _dev(out["U"], "U"),
        _dev(out["delta"], "delta"), _stream_ptr(stream))
    _check(code, "kda_prefill_debug")
    return out


def kda_decode_check_slots(slots_host, pool_size: int) -> bool:
    """True when the host slots are in range and distinct (kda_decode_check_slots)."""
    sl = torch.as_tensor(slots_host, dtype=torch.int32).contiguous()
    return _lib.kda_decode_check_slots(ctypes.c_void_p(sl.data_ptr()), sl.numel(), pool_size) == 0


# ------------------------------------------------- gated delta rule, block plan --

def _ptr(t: Optional[torch.Tensor], name: str, dtype, index: int, shape=None):
    """Address of a tensor that must be contiguous, of ``dtype`` and on CUDA device ``index``
    (and of ``shape``); None stays None."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous() and (
            shape is None or t.shape == shape):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _count(n: int, name: str) -> None:
    """A number that the C interface takes in 32 bits (it refuses negative ones itself).  The
    callers look at n >> 31 first: a call more cost the shortest operators a tenth of a microsecond."""
    if not -0x80000000 <= n <= 0x7fffffff:
        raise ValueError(f"{name} does not fit 32 bits: {n}")


def _call(fn, where: str, index: int, stream, *args):
    """One library call on device ``index``, on ``stream`` or that device's current stream."""
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        code = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            code = fn(*args, raw)
    if code != 0:
        raise KdaError(code, where)


def _gdr_device(q, k, v) -> int:
    index = q.get_device()
    if index < 0:
        raise ValueError("q must be a CUDA tensor")
    if q.dtype not in KDA_DTYPE:
        raise ValueError(f"unsupported dtype {q.dtype}")
    if k.shape != q.shape:
        raise ValueError(f"k must have q's shape {tuple(q.shape)}, got {tuple(k.shape)}")
    return index


def _pool(state, H, dk, dv, index: int):
    """Address and rows of the state pool [P, H, dk, dv]."""
    if state is None:
        return None, 0
    rows = state.shape[0]
    return _ptr(state, "state", torch.float32, index, (rows, H, dk, dv)), rows


def kda_gdr_prefill_workspace_size(total_tokens: int, num_seqs: int, Hk: int, H: int, dk: int,
                                   dv: int, dtype=torch.bfloat16, algo: str = "auto") -> int:
    return int(_lib.kda_gdr_prefill_workspace_size(total_tokens, num_seqs, Hk, H, dk, dv,
                                                   KDA_DTYPE[dtype], KDA_ALGO[algo]))


def kda_gdr_prefill(q, k, v, g, beta, cu_seqlens, cu_seqlens_host=None, state=None,
                    src_slots=None, dst_slots=None, ctx_lens=None, block_table=None,
                    block_size: int = 0, scale: float = 1.0, o=None, workspace=None,
                    algo: str = "auto", stream=None):
    """Gated delta rule (one log-decay per token and head) over packed sequences; returns o.

    q, k [T,Hk,dk], v [T,H,dv] (bf16 or fp32, one dtype), Hk dividing H; g, beta [T,H]
    fp32; cu_seqlens [N+1] int32 on the device, cu_seqlens_host an optional CPU copy.
    ``state`` [P,H,dk,dv] fp32 is a pool of state rows, updated in place: sequence n
    starts from row src_slots[n] (None, or a row outside the pool: zeros) and leaves its
    state in row dst_slots[n].  With ``block_size`` > 0 (a multiple of 64) the state after
    every completed block of ctx_lens[n] + new tokens goes to its row of ``block_table``
    [N, blocks].
    """
    if block_size >> 31:
        _count(block_size, "block_size")
    dev = _gdr_device(q, k, v)
    T, Hk, dk = q.shape
    _, H, dv = v.shape
    N = cu_seqlens.shape[0] - 1
    dt = q.dtype
    if o is None:
        o = _made(stream, torch.empty_like, v)
    host = None
    if cu_seqlens_host is not None:
        if cu_seqlens_host.numel() != N + 1 or cu_seqlens_host.device.type != "cpu":
            raise ValueError("cu_seqlens_host must be a CPU tensor of cu_seqlens' length")
        ch = cu_seqlens_host.to(torch.int32).contiguous()
        host = ch.data_ptr()
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr = _ptr(workspace, "workspace", workspace.dtype, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    pool, rows = _pool(state, H, dk, dv, dev)
    cols = block_table.shape[1] if block_table is not None else 0
    args = [_ptr(q, "q", dt, dev), _ptr(k, "k", dt, dev), _ptr(v, "v", dt, dev, (T, H, dv)),
            _ptr(g, "g", torch.float32, dev, (T, H)), _ptr(beta, "beta", torch.float32, dev, (T, H)),
            _ptr(cu_seqlens, "cu_seqlens", torch.int32, dev, (N + 1,)), host, N, T, Hk, H, dk, dv,
            KDA_DTYPE[dt], scale, pool, rows, _ptr(src_slots, "src_slots", torch.int32, dev, (N,)),
            _ptr(dst_slots, "dst_slots", torch.int32, dev, (N,)),
            _ptr(ctx_lens, "ctx_lens", torch.int32, dev, (N,)),
            _ptr(block_table, "block_table", torch.int32, dev, (N, cols)), cols, block_size,
            _ptr(o, "o", dt, dev, v.shape), ws_ptr, ws_bytes, KDA_ALGO[algo]]
    try:
        _call(_lib.kda_gdr_prefill, "kda_gdr_prefill", dev, stream, *args)
    except KdaError as e:
        if e.code != 3:            # KDA_ERR_WORKSPACE: nothing was launched
            raise
        need = kda_gdr_prefill_workspace_size(T, N, Hk, H, dk, dv, dt, algo)
        workspace = _made(stream, torch.empty, need, dtype=torch.uint8, device=q.device)
        args[-3:-1] = workspace.data_ptr(), need
        _call(_lib.kda_gdr_prefill, "kda_gdr_prefill", dev, stream, *args)
    return o


def kda_gdr_decode(q, k, v, g, beta, state, src_slots=None, dst_slots=None, num_tokens=None,
                   update_state: bool = True, scale: float = 1.0, o=None,
                   want_outputs: bool = True, stream=None, ctx_lens=None, block_table=None,
                   block_size: int = 0):
    """Gated delta rule for one or a few tokens of each sequence; returns o (or None).

    q, k [B,Hk,dk] or [B,Tq,Hk,dk], v [B,(Tq,)H,dv], g, beta [B,(Tq,)H] fp32, Tq <= 64;
    ``state`` [P,H,dk,dv] fp32 is the pool.  Sequence b reads row src_slots[b] (None: b)
    and, with ``update_state``, writes row dst_slots[b] (None: the row it read) after its
    first num_tokens[b] tokens; rows outside the pool are zeros / not written.
    ``update_state=False`` is a verify pass.  With ``block_size`` > 0 the state after every
    block of ctx_lens[b] + applied tokens that the call completes goes to its row of
    ``block_table`` [B, blocks] (kda_gdr_decode_blocks).
    """
    if block_size >> 31:
        _count(block_size, "block_size")
    dev = _gdr_device(q, k, v)
    if q.dim() == 3:
        B, Hk, dk = q.shape
        Tq, lead = 1, (B,)
    else:
        B, Tq, Hk, dk = q.shape
        lead = (B, Tq)
    H, dv = v.shape[-2:]
    dt, f32, i32 = q.dtype, torch.float32, torch.int32
    vshape, gshape, slots = (*lead, H, dv), (*lead, H), (B,)
    if o is None and (want_outputs or not update_state):
        o = _made(stream, torch.empty_like, v)
    pool, rows = _pool(state, H, dk, dv, dev)
    if block_size == 0:
        fn, where, more = _lib.kda_gdr_decode, "kda_gdr_decode", (1 if update_state else 0,)
    elif update_state:
        fn, where = _lib.kda_gdr_decode_blocks, "kda_gdr_decode_blocks"
        cols = block_table.shape[1] if block_table is not None else 0
        more = (_ptr(ctx_lens, "ctx_lens", i32, dev, slots),
                _ptr(block_table, "block_table", i32, dev, (B, cols)), cols, block_size)
    else:
        raise ValueError("block_size needs update_state: a verify pass writes no rows")
    _call(fn, where, dev, stream,
          _ptr(q, "q", dt, dev), _ptr(k, "k", dt, dev), _ptr(v, "v", dt, dev, vshape),
          _ptr(g, "g", f32, dev, gshape), _ptr(beta, "beta", f32, dev, gshape),
          B, Tq, Hk, H, dk, dv, KDA_DTYPE[dt], scale, pool, rows,
          _ptr(src_slots, "src_slots", i32, dev, slots),
          _ptr(dst_slots, "dst_slots", i32, dev, slots),
          _ptr(num_tokens, "num_tokens", i32, dev, slots), *more, _ptr(o, "o", dt, dev, vshape))
    return o


class BlockPlan(NamedTuple):
    """What kda_block_plan writes (device tensors); the block table is updated in place."""
    cu_seqlens: torch.Tensor    # [N+1] int32
    positions: torch.Tensor     # [T] int32
    token_slots: torch.Tensor   # [T] int64
    src_slots: torch.Tensor     # [N] int32
    dst_slots: torch.Tensor     # [N] int32
    free_head: torch.Tensor     # [1] int32


def kda_block_plan(new_lens, ctx_lens, free_blocks, free_head, block_table, block_size: int,
                   total_tokens: int, out: Optional[BlockPlan] = None, stream=None) -> BlockPlan:
    """Block tables and slot maps from request lengths, on the device.

    new_lens [N] int32 (tokens of this call), ctx_lens [N] int32 or None (tokens stored
    before it), free_blocks [F] int32 with free_head [1] int32 (entries from there on are
    free), block_table [N,M] int32, extended in place.  ``total_tokens`` is the length of
    the token outputs (entries past the last token are -1).  Returns a ``BlockPlan``;
    ``out`` passes its tensors (``out.free_head`` may be ``free_head`` itself).
    """
    if (block_size | total_tokens) >> 31:
        _count(block_size, "block_size")
        _count(total_tokens, "total_tokens")
    dev = new_lens.get_device()
    if dev < 0:
        raise ValueError("new_lens must be a CUDA tensor")
    (N,), (F,), i32 = new_lens.shape, free_blocks.shape, torch.int32
    if block_table.dim() != 2 or block_table.shape[0] != N:
        raise ValueError(f"block_table must have shape ({N}, blocks)")
    M = block_table.shape[1]
    if (N | F | M) >> 31:
        _count(max(N, F, M), "a length of new_lens, free_blocks or block_table")
    if total_tokens < 0:
        raise ValueError("total_tokens must not be negative")
    if out is None:
        # One allocation for the int32 outputs, padded so that the positions are 16-byte aligned.
        at = 3 * N + 2 + -(3 * N + 2) % 4
        device = new_lens.device
        if stream is None:
            flat = torch.empty(at + total_tokens, dtype=i32, device=device)
            slots = torch.empty(total_tokens, dtype=torch.int64, device=device)
        else:
            flat = _made(stream, torch.empty, at + total_tokens, dtype=i32, device=device)
            slots = _made(stream, torch.empty, total_tokens, dtype=torch.int64, device=device)
        cu, src, dst, head, _, pos = flat.split_with_sizes((N + 1, N, N, 1, at - 3 * N - 2, total_tokens))
        out = BlockPlan(cu, pos, slots, src, dst, head)
        p = flat.data_ptr()
        cu, src, dst, head, pos, slots = (p, p + 4 * (N + 1), p + 4 * (2 * N + 1), p + 4 * (3 * N + 1),
                                          p + 4 * at, slots.data_ptr())
    else:
        cu = _ptr(out.cu_seqlens, "cu_seqlens", i32, dev, (N + 1,))
        pos = _ptr(out.positions, "positions", i32, dev, (total_tokens,))
        slots = _ptr(out.token_slots, "token_slots", torch.int64, dev, (total_tokens,))
        src = _ptr(out.src_slots, "src_slots", i32, dev, (N,))
        dst = _ptr(out.dst_slots, "dst_slots", i32, dev, (N,))
        head = _ptr(out.free_head, "free_head", i32, dev, (1,))
    _call(_lib.kda_block_plan, "kda_block_plan", dev, stream,
          _ptr(new_lens, "new_lens", i32, dev, (N,)), _ptr(ctx_lens, "ctx_lens", i32, dev, (N,)),
          N, _ptr(free_blocks, "free_blocks", i32, dev, (F,)), F,
          _ptr(free_head, "free_head", i32, dev, (1,)),
          _ptr(block_table, "block_table", i32, dev), M, block_size,
          total_tokens, cu, pos, slots, src, dst, head)
    return out
