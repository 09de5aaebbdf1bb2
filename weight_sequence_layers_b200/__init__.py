"""Python binding of the B200 chunkwise-TTT library (libttt.so, C ABI in include/ttt.h).

Argument marshalling only: every function here forwards torch tensors' device pointers,
sizes and the current CUDA stream to the C entry point of the same name and raises
TTTError on a non-OK status. Every step of the computation runs in the library's CUDA
kernels; there is no fallback of any kind. (_bind.so, where it is built, makes the argument checks
of the block operators in one native call.) Importing fails loudly if libttt.so has not
been built (python weight_sequence_layers_b200/build.py).
"""
from __future__ import annotations

import ctypes
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libttt.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "ttt.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with python weight_sequence_layers_b200/build.py")

_lib = ctypes.CDLL(LIB_PATH)

(OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT,
 ERR_RANGE) = range(8)
F32, BF16 = 0, 1
LOSS = {"mse": 0, "ip": 1}
ACT = {"id": 0, "silu": 1}
DECAY = {"scalar": 0, "vector": 1}
GATE = {"decay": 0, "sigmoid": 1}


class TTTError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class ttt_config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("C", ctypes.c_int),
                ("dtype", ctypes.c_int), ("loss", ctypes.c_int), ("act", ctypes.c_int),
                ("lr_bias", ctypes.c_float), ("decay", ctypes.c_int),
                ("w0_shared", ctypes.c_int)]


class ttt_norm_config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
                ("d", ctypes.c_int), ("dtype", ctypes.c_int), ("token_major", ctypes.c_int),
                ("eps", ctypes.c_float)]


class ttt_recur_config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("gate", ctypes.c_int)]


_p, _i, _u, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_float, ctypes.c_size_t
_cfgp = ctypes.POINTER(ttt_config)
_normp, _recurp = ctypes.POINTER(ttt_norm_config), ctypes.POINTER(ttt_recur_config)
_SIGS = {
    "ttt_workspace_bytes": ([_cfgp, _i], _sz),
    "ttt_saved_bytes": ([_cfgp], _sz),
    "ttt_chunk_fwd": ([_cfgp] + [_p] * 11 + [_sz, _p], _i),
    "ttt_chunk_bwd": ([_cfgp] + [_p] * 19 + [_sz, _p], _i),
    "inplace_ttt_workspace_bytes": ([_i] * 4, _sz),
    "ttt_mlp_workspace_bytes": ([_cfgp, _i], _sz),
    "ttt_mlp_fwd": ([_cfgp, _i] + [_p] * 13 + [_sz, _p], _i),
    "ttt_mlp_bwd": ([_cfgp, _i] + [_p] * 17 + [_sz, _p], _i),
    "inplace_ttt_fwd": ([_i] * 4 + [_f] + [_p] * 6 + [_sz, _p], _i),
    "inplace_ttt_bwd": ([_i] * 4 + [_f] + [_p] * 9 + [_sz, _p], _i),
    "inplace_ttt_target_workspace_bytes": ([_i] * 2, _sz),
    "inplace_ttt_docs_workspace_bytes": ([_i] * 4, _sz),
    "inplace_ttt_delta": ([_i] * 3 + [_f] + [_p] * 4 + [_sz, _p], _i),
    "ttt_add_f32": ([_p, _p, _sz, _p], _i),
    "inplace_ttt_fwd_docs": ([_i] * 4 + [_f] + [_p] * 6 + [_i, _p, _sz, _p], _i),
    "inplace_ttt_bwd_docs": ([_i] * 4 + [_f] + [_p] * 9 + [_i, _p, _sz, _p], _i),
    "inplace_ttt_target": ([_i] * 3 + [_p] * 5 + [_sz, _p], _i),
    "inplace_ttt_target_bwd_workspace_bytes": ([_i] * 3, _sz),
    "inplace_ttt_target_bwd": ([_i] * 3 + [_p] * 8 + [_sz, _p], _i),
    "ttt_norm_fwd": ([_normp] + [_p] * 9, _i),
    "ttt_norm_bwd_workspace_bytes": ([_normp], _sz),
    "ttt_norm_bwd": ([_normp] + [_p] * 10 + [_sz, _p], _i),
    "ttt_recur_fwd": ([_recurp] + [_p] * 7, _i),
    "ttt_recur_bwd": ([_recurp] + [_p] * 11, _i),
    "ttt_recur_step": ([_recurp] + [_p] * 3 + [_i] + [_p] * 3, _i),
    "ttt_linear_workspace_bytes": ([_i] * 4, _sz),
    "ttt_linear_fwd": ([_i] * 4 + [_p] * 8 + [_sz, _p], _i),
    "ttt_linear_bwd": ([_i] * 4 + [_p] * 10 + [_sz, _p], _i),
    "ttt_get_device_error": ([_p], _i),
    "ttt_selftest_bounded_wait": ([_u, _p], _i),
    "ttt_status_string": ([_i], ctypes.c_char_p),
    "ttt_kernel_launches": ([], ctypes.c_ulonglong),
    "ttt_chunk_bwd_noalloc": ([_cfgp] + [_p] * 18 + [_p], _i),
}
for _name, (_args, _ret) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _ret


def header_functions() -> list[str]:
    """Names of the functions include/ttt.h declares."""
    text = open(HEADER).read()
    # a declaration starts in column 0 with its return type (one or more words, pointers
    # included), then the name and "("; comments, macros and continuation lines do not
    return re.findall(r"^(?!typedef\b)(?:[A-Za-z_]\w*[ \t\*]+)+([A-Za-z_]\w*)\s*\(", text,
                      flags=re.M)


def status_string(status: int) -> str:
    return _lib.ttt_status_string(int(status)).decode()


def _ptr(t):
    """Device address of a tensor argument; None and raw integer addresses pass through.

    The library reads and writes every array argument as a dense row-major array on the
    current CUDA device. A strided view, a host tensor or a tensor on another device would
    give wrong results or a memory fault, so they are refused here, before any library call.
    """
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (dense row-major, no strided views)")
    if not t.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors: the library takes device pointers")
    import torch
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensor on {t.device}, but the library runs on the current device "
                         f"cuda:{torch.cuda.current_device()}")
    return t.data_ptr()


_modules = []  # torch and the native argument checks, on first use: torch loads slowly


def _torch():
    if not _modules:
        import torch
        try:
            from . import _bind
        except ImportError:  # not built: every check is made below, in Python
            _bind = None
        _modules.extend((torch, _bind))
    return _modules[0]


def _stream(stream):
    if stream is None:
        torch = _torch()
        if torch.cuda.is_initialized():
            # current_stream() builds a Stream object: 3.4 us, a quarter of a small call
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != OK:
        raise TTTError(status, where)


def make_config(B, H, T, dk, dv, C, dtype="bf16", loss="mse", act="id", lr_bias=0.0,
                decay="scalar", w0_shared=False) -> ttt_config:
    """decay: "scalar" (gamma [B,H,T], or no gamma) or "vector" (gamma [B,H,T,dk]).
    w0_shared: W0 (W1_0, W2_0 for TTT-MLP) is [H, ...], one initial state per head shared by
    the batch, instead of [B, H, ...]."""
    return ttt_config(B, H, T, dk, dv, C, F32 if dtype in ("f32", F32) else BF16,
                      LOSS.get(loss, loss), ACT.get(act, act), float(lr_bias),
                      DECAY.get(decay, decay), int(bool(w0_shared)))


def ttt_saved_bytes(cfg: ttt_config) -> int:
    """Bytes of the forward's G_saved buffer (G, and Zq with SiLU)."""
    n = _lib.ttt_saved_bytes(ctypes.byref(cfg))
    if n == ctypes.c_size_t(-1).value:
        raise TTTError(ERR_INVALID_ARG, "ttt_saved_bytes")
    return n


def ttt_workspace_bytes(cfg: ttt_config, for_bwd: int) -> int:
    """for_bwd: 0 forward, 1 backward without G_saved, 2 backward given G_saved."""
    n = _lib.ttt_workspace_bytes(ctypes.byref(cfg), int(for_bwd))
    if n == ctypes.c_size_t(-1).value:
        raise TTTError(ERR_INVALID_ARG, "ttt_workspace_bytes")
    return n


def _check_size(t, nbytes: int, name: str):
    """A buffer the library fills or reads for this config must hold nbytes; the C ABI cannot
    tell, and a short buffer would be written past its end."""
    if t is not None and not isinstance(t, int) and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, the config needs "
                         f"{nbytes}")


def _chunks_bytes(cfg) -> int:
    return cfg.B * cfg.H * (cfg.T // cfg.C) * cfg.dk * cfg.dv * (2 if cfg.dtype == BF16 else 4)


def ttt_chunk_fwd(cfg, Q, K, V, beta, gamma, W0, O, W_final=None, W_chunks=None, G_saved=None,
                  workspace=None, workspace_bytes=0, stream=None):
    """Forward of the chunkwise TTT layer on the current device and stream.

    Q, K [B,H,T,dk]; V, O [B,H,T,dv] in cfg's dtype; beta [B,H,T] and W0, W_final [B,H,dk,dv]
    float32; gamma [B,H,T] or [B,H,T,dk] float32, or None (no decay). W_chunks
    [B,H,T/C,dk,dv] in cfg's dtype and G_saved (ttt_saved_bytes) are optional outputs that
    ttt_chunk_bwd reads. Workspace: ttt_workspace_bytes(cfg, 0) bytes. Raises TTTError on a
    non-OK status."""
    if G_saved is not None:
        _check_size(G_saved, ttt_saved_bytes(cfg), "G_saved")
    if W_chunks is not None:
        _check_size(W_chunks, _chunks_bytes(cfg), "W_chunks")
    st = _lib.ttt_chunk_fwd(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(beta), _ptr(gamma),
                            _ptr(W0), _ptr(O), _ptr(W_final), _ptr(W_chunks), _ptr(G_saved),
                            _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "ttt_chunk_fwd")


def ttt_chunk_bwd(cfg, Q, K, V, beta, gamma, W0, W_chunks, G_saved, dO, dW_final, O, W_final, dQ,
                  dK, dV, dbeta, dW0, dgamma, workspace=None, workspace_bytes=0, stream=None):
    """Analytic backward of the layer for J = <dO, O> + <dW_final, W_final>.

    Takes the forward's inputs, its W_chunks and (optionally) G_saved, dO and dW_final (or
    None), and writes dQ, dK, dV, dbeta, dW0 and, when dgamma is given, the decay gradient
    (which also needs the forward's O, and W_final when dW_final is given). Workspace:
    ttt_workspace_bytes(cfg, 2 if G_saved is passed else 1) bytes."""
    if G_saved is not None:
        _check_size(G_saved, ttt_saved_bytes(cfg), "G_saved")
    st = _lib.ttt_chunk_bwd(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(beta), _ptr(gamma),
                            _ptr(W0), _ptr(W_chunks), _ptr(G_saved), _ptr(dO), _ptr(dW_final),
                            _ptr(O), _ptr(W_final), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dbeta),
                            _ptr(dW0), _ptr(dgamma), _ptr(workspace), int(workspace_bytes),
                            _stream(stream))
    _check(st, "ttt_chunk_bwd")


NOALLOC_SCRATCH_BYTES = 8 << 20


def ttt_chunk_bwd_noalloc(cfg, Q, K, V, beta, gamma, W0, W_chunks, G_saved, dO, dW_final, O,
                          W_final, dQ, dK, dV, dbeta, dW0, dgamma, stream=None):
    """ttt_chunk_bwd for callers that cannot allocate: scratch is the library's fixed array."""
    if G_saved is not None:
        _check_size(G_saved, ttt_saved_bytes(cfg), "G_saved")
    st = _lib.ttt_chunk_bwd_noalloc(ctypes.byref(cfg), _ptr(Q), _ptr(K), _ptr(V), _ptr(beta),
                                    _ptr(gamma), _ptr(W0), _ptr(W_chunks), _ptr(G_saved),
                                    _ptr(dO), _ptr(dW_final), _ptr(O), _ptr(W_final), _ptr(dQ),
                                    _ptr(dK), _ptr(dV), _ptr(dbeta), _ptr(dW0), _ptr(dgamma),
                                    _stream(stream))
    _check(st, "ttt_chunk_bwd_noalloc")


def ttt_mlp_workspace_bytes(cfg: ttt_config, hidden: int) -> int:
    n = _lib.ttt_mlp_workspace_bytes(ctypes.byref(cfg), int(hidden))
    if n == ctypes.c_size_t(-1).value:
        raise TTTError(ERR_INVALID_ARG, "ttt_mlp_workspace_bytes")
    return n


def ttt_mlp_fwd(cfg, hidden, Q, K, V, beta, gamma, W1_0, W2_0, O, W1_final, W2_final, W1_chunks,
                W2_chunks, workspace, workspace_bytes, stream=None):
    """TTT-MLP forward: the fast weight act(k W1) W2 with W1 [B,H,dk,hidden] and W2
    [B,H,hidden,dv] float32; W1_chunks / W2_chunks keep the chunk-start weights for the
    backward. Workspace: ttt_mlp_workspace_bytes(cfg, hidden)."""
    st = _lib.ttt_mlp_fwd(ctypes.byref(cfg), int(hidden), _ptr(Q), _ptr(K), _ptr(V), _ptr(beta),
                          _ptr(gamma), _ptr(W1_0), _ptr(W2_0), _ptr(O), _ptr(W1_final),
                          _ptr(W2_final), _ptr(W1_chunks), _ptr(W2_chunks), _ptr(workspace),
                          int(workspace_bytes), _stream(stream))
    _check(st, "ttt_mlp_fwd")


def ttt_mlp_bwd(cfg, hidden, Q, K, V, beta, gamma, W1_chunks, W2_chunks, dO, dW1_final, dW2_final,
                dQ, dK, dV, dbeta, dW1_0, dW2_0, workspace, workspace_bytes, stream=None):
    """TTT-MLP backward for J = <dO, O> + <dW1_final, W1_final> + <dW2_final, W2_final>."""
    st = _lib.ttt_mlp_bwd(ctypes.byref(cfg), int(hidden), _ptr(Q), _ptr(K), _ptr(V), _ptr(beta),
                          _ptr(gamma), _ptr(W1_chunks), _ptr(W2_chunks), _ptr(dO), _ptr(dW1_final),
                          _ptr(dW2_final), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dbeta), _ptr(dW1_0),
                          _ptr(dW2_0), _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "ttt_mlp_bwd")


def inplace_ttt_workspace_bytes(T, d_ff, d_model, C) -> int:
    n = _lib.inplace_ttt_workspace_bytes(T, d_ff, d_model, C)
    if n == ctypes.c_size_t(-1).value:
        raise TTTError(ERR_INVALID_ARG, "inplace_ttt_workspace_bytes")
    return n


def inplace_ttt_fwd(T, d_ff, d_model, C, lr, Z, Vhat, W, O, workspace=None, workspace_bytes=0,
                    stream=None, W_chunks=None):
    """In-Place TTT forward: per chunk of C tokens O_i = Z_i W^T, then W += lr Vhat_i^T Z_i.

    Z [T,d_ff] and Vhat [T,d_model] bf16; W [d_model,d_ff] float32 in/out; O [T,d_model] bf16;
    W_chunks [T/C,d_model,d_ff] bf16 (optional) keeps the weight each chunk applied, for
    inplace_ttt_bwd. Workspace: inplace_ttt_workspace_bytes(T, d_ff, d_model, C)."""
    st = _lib.inplace_ttt_fwd(T, d_ff, d_model, C, float(lr), _ptr(Z), _ptr(Vhat), _ptr(W),
                              _ptr(O), _ptr(W_chunks), _ptr(workspace), int(workspace_bytes),
                              _stream(stream))
    _check(st, "inplace_ttt_fwd")


def _int_array(xs):
    xs = [int(x) for x in xs]
    return (ctypes.c_int * max(1, len(xs)))(*xs), len(xs)


def inplace_ttt_docs_workspace_bytes(T, d_ff, d_model, C) -> int:
    n = _lib.inplace_ttt_docs_workspace_bytes(T, d_ff, d_model, C)
    if n == ctypes.c_size_t(-1).value:
        raise TTTError(ERR_INVALID_ARG, "inplace_ttt_docs_workspace_bytes")
    return n


def inplace_ttt_fwd_docs(T, d_ff, d_model, C, lr, Z, Vhat, W, O, W_chunks, doc_starts, workspace,
                         workspace_bytes, stream=None):
    arr, n = _int_array(doc_starts)
    st = _lib.inplace_ttt_fwd_docs(T, d_ff, d_model, C, float(lr), _ptr(Z), _ptr(Vhat), _ptr(W),
                                   _ptr(O), _ptr(W_chunks), arr, n, _ptr(workspace),
                                   int(workspace_bytes), _stream(stream))
    _check(st, "inplace_ttt_fwd_docs")


def inplace_ttt_bwd_docs(T, d_ff, d_model, C, lr, Z, Vhat, W_chunks, dO, dW_final, dZ, dVhat, dW,
                         doc_starts, workspace, workspace_bytes, stream=None):
    arr, n = _int_array(doc_starts)
    st = _lib.inplace_ttt_bwd_docs(T, d_ff, d_model, C, float(lr), _ptr(Z), _ptr(Vhat),
                                   _ptr(W_chunks), _ptr(dO), _ptr(dW_final), _ptr(dZ), _ptr(dVhat),
                                   _ptr(dW), arr, n, _ptr(workspace), int(workspace_bytes),
                                   _stream(stream))
    _check(st, "inplace_ttt_bwd_docs")


def inplace_ttt_target_workspace_bytes(T, d_model) -> int:
    n = _lib.inplace_ttt_target_workspace_bytes(T, d_model)
    if n == ctypes.c_size_t(-1).value:
        raise TTTError(ERR_INVALID_ARG, "inplace_ttt_target_workspace_bytes")
    return n


def inplace_ttt_target(T, d_model, k, X0, conv_w, W_target, Vhat, workspace=None,
                       workspace_bytes=0, stream=None):
    st = _lib.inplace_ttt_target(T, d_model, k, _ptr(X0), _ptr(conv_w), _ptr(W_target), _ptr(Vhat),
                                 _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "inplace_ttt_target")


def inplace_ttt_target_bwd_workspace_bytes(T, d_model, k) -> int:
    n = _lib.inplace_ttt_target_bwd_workspace_bytes(T, d_model, k)
    if n == ctypes.c_size_t(-1).value:
        raise TTTError(ERR_INVALID_ARG, "inplace_ttt_target_bwd_workspace_bytes")
    return n


def inplace_ttt_target_bwd(T, d_model, k, X0, conv_w, W_target, dVhat, dX0, dconv_w, dW_target,
                           workspace=None, workspace_bytes=0, stream=None):
    st = _lib.inplace_ttt_target_bwd(T, d_model, k, _ptr(X0), _ptr(conv_w), _ptr(W_target),
                                     _ptr(dVhat), _ptr(dX0), _ptr(dconv_w), _ptr(dW_target),
                                     _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "inplace_ttt_target_bwd")


def inplace_ttt_bwd(T, d_ff, d_model, C, lr, Z, Vhat, W_chunks, dO, dW_final, dZ, dVhat, dW,
                    workspace=None, workspace_bytes=0, stream=None):
    """In-Place TTT backward for J = sum_i <dO_i, O_i> + <dW_final, W_final> (dW_final may
    be None): writes dZ [T,d_ff] and dVhat [T,d_model] bf16 and dW, the float32 gradient of the
    initial W, from the forward's W_chunks."""
    st = _lib.inplace_ttt_bwd(T, d_ff, d_model, C, float(lr), _ptr(Z), _ptr(Vhat), _ptr(W_chunks),
                              _ptr(dO), _ptr(dW_final), _ptr(dZ), _ptr(dVhat), _ptr(dW),
                              _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "inplace_ttt_bwd")


def ttt_get_device_error(stream=None) -> int:
    """Returns the status (OK, ERR_TIMEOUT, ERR_RANGE or ERR_CUDA) instead of raising."""
    return _lib.ttt_get_device_error(_stream(stream))


def ttt_selftest_bounded_wait(spin_limit: int, stream=None):
    _check(_lib.ttt_selftest_bounded_wait(int(spin_limit), _stream(stream)), "ttt_selftest_bounded_wait")


def ttt_kernel_launches() -> int:
    return int(_lib.ttt_kernel_launches())


# Raw C entry points (for callers that marshal pointers themselves).
lib = _lib


def inplace_ttt_delta(T, d_ff, d_model, lr, Z, Vhat, dW, workspace, workspace_bytes, stream=None):
    """dW = lr Vhat^T Z over all T tokens (the summed chunk updates of one shard)."""
    st = _lib.inplace_ttt_delta(T, d_ff, d_model, float(lr), _ptr(Z), _ptr(Vhat), _ptr(dW),
                                _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "inplace_ttt_delta")


def ttt_add_f32(dst, src, stream=None):
    st = _lib.ttt_add_f32(_ptr(dst), _ptr(src), int(dst.numel()), _stream(stream))
    _check(st, "ttt_add_f32")


class _CudaOps:
    """The library calls the context-parallel In-Place forward is made of."""

    @staticmethod
    def delta(T, d_ff, d_model, lr, Z, Vhat, dW, workspace, workspace_bytes):
        inplace_ttt_delta(T, d_ff, d_model, lr, Z, Vhat, dW, workspace, workspace_bytes)

    @staticmethod
    def add(dst, src):
        ttt_add_f32(dst, src)

    @staticmethod
    def fwd(T, d_ff, d_model, C, lr, Z, Vhat, W, O, workspace, workspace_bytes):
        inplace_ttt_fwd(T, d_ff, d_model, C, lr, Z, Vhat, W, O, workspace, workspace_bytes)


def inplace_cp_fwd(T, d_ff, d_model, C, lr, Z, Vhat, W, O, workspace, workspace_bytes,
                   group=None, ops=None):
    """Context-parallel In-Place forward (page "In-Place Test-Time Training", section "核心方法和
    技术细节": the update is associative, so the chunk loop runs as a parallel scan across
    devices). The sequence is split in order across the ranks of `group`; this rank holds its
    T tokens (Z [T, d_ff], Vhat [T, d_model]), and W holds the initial W_down on every rank.
    Each rank computes its shard's summed update dW_g = lr Vhat_g^T Z_g, the ranks exchange
    them (all-gather), rank g adds dW_h for h < g to W and runs inplace_ttt_fwd on its tokens.
    On return O holds this shard's outputs and W its end state (the last rank's W is the
    sequence's final W_down). `ops` replaces the library calls (the CPU tests of the exchange
    pass an implementation built on the oracle); by default they are the C ABI's."""
    import torch
    import torch.distributed as dist
    ops = ops or _CudaOps
    world = dist.get_world_size(group)
    rank = dist.get_rank(group)
    dW = torch.empty_like(W)
    ops.delta(T, d_ff, d_model, lr, Z, Vhat, dW, workspace, workspace_bytes)
    parts = [torch.empty_like(dW) for _ in range(world)]
    dist.all_gather(parts, dW, group=group)
    for h in range(rank):
        ops.add(W, parts[h])
    ops.fwd(T, d_ff, d_model, C, lr, Z, Vhat, W, O, workspace, workspace_bytes)


def _tensors(where, *specs):
    """Device addresses of the tensor arguments (name, tensor, elements, dtype) of one call.

    Like _ptr, and each tensor must have the dtype and the number of elements that the call's
    sizes give it: the C ABI sees addresses only, and a short buffer would be read or written
    past its end. None and raw integer addresses pass through unchecked."""
    dev, out = -1, []
    for name, t, n, dtype in specs:
        if t is None or isinstance(t, int):
            out.append(t)
            continue
        if t.dtype is not dtype or t.numel() != n:
            raise ValueError(f"{where}: {name} is {t.numel()} x {t.dtype}, expected {n} x {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous (dense row-major)")
        at = t.get_device()
        if at != dev or at < 0:
            if not t.is_cuda:
                raise ValueError(f"{where}: {name} must be a CUDA tensor")
            import torch
            dev = torch.cuda.current_device()
            if at != dev:
                raise ValueError(f"{where}: {name} is on {t.device}, but the library runs on the "
                                 f"current device cuda:{dev}")
        out.append(t.data_ptr())
    return out


def _ptrs(where, names, tensors, counts, kinds):
    """_tensors with the types as a string (b bfloat16, f float32, i int32, u uint8), by the native
    checks where all is well (0.5 us for eight tensors against 4)."""
    torch = _torch()
    if _modules[1] is not None and torch.cuda.is_initialized():
        p = _modules[1].ptrs(tensors, counts, kinds, torch._C._cuda_getDevice())
        if p is not None:
            return p
    types = {"b": torch.bfloat16, "f": torch.float32, "i": torch.int32, "u": torch.uint8}
    return _tensors(where, *zip(names, tensors, counts, (types[k] for k in kinds)))


def _kind(code):
    return "b" if code == BF16 else "f"


def make_norm_config(B, H, T, d, dtype="bf16", token_major=False, eps=1e-5) -> ttt_norm_config:
    """Rows of d features, B * H * T of them, with one weight row per head (H = 1: the plain
    layer norm). token_major: Y and dY are [B, T, H, d] instead of [B, H, T, d]."""
    return ttt_norm_config(B, H, T, d, F32 if dtype in ("f32", F32) else BF16,
                           int(bool(token_major)), float(eps))


def ttt_norm_fwd(cfg, X, residual, weight, bias, Y, S=None, mean=None, rstd=None, stream=None):
    """Layer norm forward: s = X + residual (X when residual is None), Y = norm(s) * weight +
    bias, S = s. X, residual, S [B,H,T,d] and Y ([B,T,H,d] if cfg.token_major) in cfg's dtype;
    weight, bias [H,d] and mean, rstd [B,H,T] float32. residual, weight, bias, S, mean and rstd
    may be None."""
    k, rows, hd = _kind(cfg.dtype), cfg.B * cfg.H * cfg.T, cfg.H * cfg.d
    n = rows * cfg.d
    p = _ptrs("ttt_norm_fwd", ("X", "residual", "weight", "bias", "Y", "S", "mean", "rstd"),
              (X, residual, weight, bias, Y, S, mean, rstd), (n, n, hd, hd, n, n, rows, rows),
              k + k + "ff" + k + k + "ff")
    _check(_lib.ttt_norm_fwd(ctypes.byref(cfg), *p, _stream(stream)), "ttt_norm_fwd")


def ttt_norm_bwd_workspace_bytes(cfg) -> int:
    n = _lib.ttt_norm_bwd_workspace_bytes(ctypes.byref(cfg))
    if n == ctypes.c_size_t(-1).value:
        raise TTTError(ERR_INVALID_ARG, "ttt_norm_bwd_workspace_bytes")
    return n


def ttt_norm_bwd(cfg, S, weight, mean, rstd, dY, dS, dX, dweight=None, dbias=None, workspace=None,
                 workspace_bytes=0, stream=None):
    """Layer norm backward for J = <dY, Y> + <dS, S> (dS may be None): dX (the gradient of X and
    of residual), dweight and dbias [H,d] float32 (each may be None). S is the forward's S, or
    its X without a residual. Workspace: ttt_norm_bwd_workspace_bytes(cfg)."""
    k, rows, hd = _kind(cfg.dtype), cfg.B * cfg.H * cfg.T, cfg.H * cfg.d
    n = rows * cfg.d
    p = _ptrs("ttt_norm_bwd",
              ("S", "weight", "mean", "rstd", "dY", "dS", "dX", "dweight", "dbias"),
              (S, weight, mean, rstd, dY, dS, dX, dweight, dbias),
              (n, hd, rows, rows, n, n, n, hd, hd), k + "fff" + k + k + k + "ff")
    _check(_lib.ttt_norm_bwd(ctypes.byref(cfg), *p, _ws(workspace, workspace_bytes),
                             int(workspace_bytes), _stream(stream)), "ttt_norm_bwd")


def _ws(t, nbytes):
    """Address of a workspace tensor that must hold the bytes the caller says it does."""
    _check_size(t, nbytes, "workspace")
    return _ptr(t)


def make_recur_config(B, T, D, dtype="bf16", gate="sigmoid") -> ttt_recur_config:
    """gate: "sigmoid" (G holds logits in dtype, u = (1 - a) X) or "decay" (G holds the decay
    itself, float32, u = X)."""
    return ttt_recur_config(B, T, D, F32 if dtype in ("f32", F32) else BF16, GATE.get(gate, gate))


def ttt_recur_fwd(cfg, X, G, reset, h0, H, h_final=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t over [B,T,D]. reset [B,T] uint8 (a nonzero
    byte starts a document: the state before that token counts as 0) and h0 [B,D] float32 may be
    None; H [B,T,D] holds every h_t, h_final [B,D] float32 (or None) the last."""
    k, n, bd = _kind(cfg.dtype), cfg.B * cfg.T * cfg.D, cfg.B * cfg.D
    p = _ptrs("ttt_recur_fwd", ("X", "G", "reset", "h0", "H", "h_final"),
              (X, G, reset, h0, H, h_final), (n, n, cfg.B * cfg.T, bd, n, bd),
              k + (k if cfg.gate else "f") + "uf" + k + "f")
    _check(_lib.ttt_recur_fwd(ctypes.byref(cfg), *p, _stream(stream)), "ttt_recur_fwd")


def ttt_recur_bwd(cfg, X, G, reset, h0, H, dH, dh_final, dX, dG, dh0=None, stream=None):
    """Backward of ttt_recur_fwd for J = <dH, H> + <dh_final, h_final>, from the forward's inputs
    and its H: dX, dG [B,T,D] in the types of X and G, dh0 [B,D] float32. reset, h0, dh_final and
    dh0 may be None, and X with the "decay" gate."""
    k, n, bd = _kind(cfg.dtype), cfg.B * cfg.T * cfg.D, cfg.B * cfg.D
    gk = k if cfg.gate else "f"
    p = _ptrs("ttt_recur_bwd",
              ("X", "G", "reset", "h0", "H", "dH", "dh_final", "dX", "dG", "dh0"),
              (X, G, reset, h0, H, dH, dh_final, dX, dG, dh0),
              (n, n, cfg.B * cfg.T, bd, n, n, bd, n, n, bd),
              k + gk + "uf" + k + k + "f" + k + gk + "f")
    _check(_lib.ttt_recur_bwd(ctypes.byref(cfg), *p, _stream(stream)), "ttt_recur_bwd")


def ttt_recur_step(cfg, X, G, slots, state, Y, stream=None):
    """One token of cfg.B rows (cfg.T = 1) against the state cache [n_slots, D] float32, updated
    in place: row b reads and writes state[slots[b]] and Y[b] is the new state. slots [B] int32
    on the device, negative for a padding row (left untouched); None: row b has slot b."""
    n_slots = state.shape[0]
    k, n = _kind(cfg.dtype), cfg.B * cfg.D
    p = _ptrs("ttt_recur_step", ("X", "G", "slots", "state", "Y"), (X, G, slots, state, Y),
              (n, n, cfg.B, n_slots * cfg.D, n), k + (k if cfg.gate else "f") + "if" + k)
    _check(_lib.ttt_recur_step(ctypes.byref(cfg), p[0], p[1], p[2], n_slots, p[3], p[4],
                               _stream(stream)), "ttt_recur_step")


def ttt_linear_workspace_bytes(M, N, K, for_bwd) -> int:
    n = _lib.ttt_linear_workspace_bytes(M, N, K, int(for_bwd))
    if n == ctypes.c_size_t(-1).value:
        raise TTTError(ERR_INVALID_ARG, "ttt_linear_workspace_bytes")
    return n


def ttt_linear_fwd(M, N, K, act, X, W, bias, mul, residual, Y, P=None, workspace=None,
                   workspace_bytes=0, stream=None):
    """Y = act(X W^T + bias) * mul + residual with act "id" or "silu". X [M,K], W [N,K] (a torch
    Linear's weight), mul, residual, Y and P [M,N] bf16, bias [N] float32; bias, mul, residual
    and P may be None. P receives X W^T + bias, which ttt_linear_bwd reads. N and K are multiples
    of 8. Workspace: ttt_linear_workspace_bytes(M, N, K, 0)."""
    mn = M * N
    p = _ptrs("ttt_linear_fwd", ("X", "W", "bias", "mul", "residual", "Y", "P"),
              (X, W, bias, mul, residual, Y, P), (M * K, N * K, N, mn, mn, mn, mn), "bbfbbbb")
    _check(_lib.ttt_linear_fwd(M, N, K, ACT.get(act, act), *p, _ws(workspace, workspace_bytes),
                               int(workspace_bytes), _stream(stream)), "ttt_linear_fwd")


def ttt_linear_bwd(M, N, K, act, X, W, P, mul, dY, dX=None, dW=None, dbias=None, dmul=None,
                   workspace=None, workspace_bytes=0, stream=None):
    """Backward of ttt_linear_fwd for J = <dY, Y>: dX [M,K], dW [N,K], dmul [M,N] bf16 and dbias
    [N] float32, each written when given (the gradient of residual is dY). P is the forward's P;
    it may be None for act "id" without mul. Workspace: ttt_linear_workspace_bytes(M, N, K, 1)."""
    mk, nk, mn = M * K, N * K, M * N
    p = _ptrs("ttt_linear_bwd", ("X", "W", "P", "mul", "dY", "dX", "dW", "dbias", "dmul"),
              (X, W, P, mul, dY, dX, dW, dbias, dmul), (mk, nk, mn, mn, mn, mk, nk, N, mn),
              "bbbbbbbfb")
    _check(_lib.ttt_linear_bwd(M, N, K, ACT.get(act, act), *p, _ws(workspace, workspace_bytes),
                               int(workspace_bytes), _stream(stream)), "ttt_linear_bwd")
