"""ctypes binding of liblmhead.so: the calls of include/lmhead.h.

Argument marshalling only: shapes, dtypes and device pointers are read off
torch tensors and passed to the C ABI on the caller's current CUDA stream.
All arithmetic happens in the library's kernels.  If the library is missing
or cannot be loaded, every call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblmhead.so")

LMH_OK, LMH_ERR_INVALID_ARG, LMH_ERR_MISALIGNED, LMH_ERR_UNSUPPORTED, LMH_ERR_CUDA = range(5)
F32, BF16, F16 = 0, 1, 2
DEV_BAD_TARGET = 0x1
DEV_PIPE_TIMEOUT = 0x2
DEV_BAD_LOGIT = 0x4
DEV_BAD_ADAPTER = 0x8
DEV_BAD_PARENT = 0x10
IGNORE_INDEX = -100

EXPORTS = ("lmhead_fwd", "ce_fwd", "ce_bwd", "lmhead_bwd_dx", "lmhead_bwd_dw",
           "lmhead_fwd_ce", "lmhead_fwd_ce_workspace_bytes", "lmhead_fwd_ce_noalloc",
           "lmhead_bwd_dw_acc", "ce_fwd_shard", "ce_merge_shards", "ce_bwd_shard",
           "lmh_status_string", "lmh_version", "lmh_watchdog_selftest",
           "lmh_gemm_watchdog_selftest", "beam_select", "beam_select_workspace_bytes",
           "beam_reorder", "lmhead_fwd_lora", "lmhead_lora_workspace_bytes", "lmhead_bwd_dx_lora",
           "lmhead_bwd_lora")

_lib = None


class LmhError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


def lib() -> ctypes.CDLL:
    """Load liblmhead.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"liblmhead.so not found at {LIB_PATH}; build it with "
                               "`python -m lm_head_fp32_b200.build` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.lmhead_fwd.argtypes = [P, P, P, I32, I64, I64, I64, P, P]
        L.ce_fwd.argtypes = [P, P, P, I64, I64, I64, P, P]
        L.ce_bwd.argtypes = [P, P, P, P, I64, P, I32, I64, I64, I64, P, P]
        L.lmhead_bwd_dx.argtypes = [P, P, P, I32, I64, I64, I64, P, P]
        L.lmhead_bwd_dw.argtypes = [P, P, P, I32, I64, I64, I64, P, P]
        for f in ("lmhead_fwd", "ce_fwd", "ce_bwd", "lmhead_bwd_dx", "lmhead_bwd_dw"):
            getattr(L, f).restype = ctypes.c_int
        L.lmh_status_string.argtypes = [ctypes.c_int]
        L.lmh_status_string.restype = ctypes.c_char_p
        L.lmh_version.restype = ctypes.c_int32
        L.lmhead_fwd_ce.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, I64, P, P]
        L.lmhead_fwd_ce.restype = ctypes.c_int
        L.ce_fwd_shard.argtypes = [P, P, P, I64, I64, I64, I64, I64, P, P]
        L.ce_merge_shards.argtypes = [P, I64, P, P, I64, I64, I64, P, P]
        L.ce_bwd_shard.argtypes = [P, P, P, P, I64, P, I32, I64, I64, I64, I64, I64, P, P]
        for f in ("ce_fwd_shard", "ce_merge_shards", "ce_bwd_shard"):
            getattr(L, f).restype = ctypes.c_int
        L.lmhead_bwd_dw_acc.argtypes = [P, P, P, I64, I64, I64, P, P]
        L.lmhead_bwd_dw_acc.restype = ctypes.c_int
        L.lmhead_fwd_ce_noalloc.argtypes = [P, P, P, P, P, I64, I64, I64, I64, P, P]
        L.lmhead_fwd_ce_noalloc.restype = ctypes.c_int
        L.lmhead_fwd_ce_workspace_bytes.argtypes = [I64, I64]
        L.lmhead_fwd_ce_workspace_bytes.restype = I64
        L.lmh_watchdog_selftest.argtypes = [P, I64, P]
        L.lmh_watchdog_selftest.restype = ctypes.c_int
        L.lmh_gemm_watchdog_selftest.argtypes = [P, P, P, I64, I64, I64, I64, P, P]
        L.lmh_gemm_watchdog_selftest.restype = ctypes.c_int
        L.beam_select.argtypes = [P, I32, P, P, P, P, P, P, P, P, P, I64, I64, I64, I64, I64, I64, P, P]
        L.beam_select_workspace_bytes.argtypes = [I64, I64, I64, I64]
        L.beam_select_workspace_bytes.restype = I64
        L.beam_reorder.argtypes = [P, I64, P, I64, I64, I64, I64, I64, P, P, I64, P, P]
        L.lmhead_lora_workspace_bytes.argtypes = [I64] * 5
        L.lmhead_lora_workspace_bytes.restype = I64
        for f in ("lmhead_fwd_lora", "lmhead_bwd_dx_lora"):
            getattr(L, f).argtypes = [P] * 8 + [I32, P] + [I64] * 6 + [P, P]
        L.lmhead_bwd_lora.argtypes = [P] * 8 + [I64] * 6 + [P, P]
        for f in ("beam_select", "beam_reorder", "lmhead_fwd_lora", "lmhead_bwd_dx_lora",
                  "lmhead_bwd_lora"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().lmh_status_string(int(code)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return F32
    if dt == torch.bfloat16:
        return BF16
    if dt == torch.float16:
        return F16          # passed through so that the library rejects it
    raise TypeError(f"unsupported dtype {dt}")


def _check(code: int, where: str):
    if code != LMH_OK:
        raise LmhError(code, where)


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous (row-major)")


def lmhead_fwd(X: torch.Tensor, W: torch.Tensor, logits: torch.Tensor,
               status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """logits[M,V] (FP32 or BF16) = X[M,K] . W[V,K]^T."""
    _contig(X, W, logits)
    M, K = X.shape
    V = W.shape[0]
    assert W.shape[1] == K and tuple(logits.shape) == (M, V)
    _check(lib().lmhead_fwd(_ptr(X), _ptr(W), _ptr(logits), _dtype_code(logits.dtype),
                            M, K, V, _ptr(status), _stream(stream)), "lmhead_fwd")
    return logits


def ce_fwd(logits: torch.Tensor, target: torch.Tensor, stats: torch.Tensor,
           ignore_index: int = IGNORE_INDEX, status: Optional[torch.Tensor] = None,
           stream=None) -> torch.Tensor:
    """stats[M,4] = {m, d, x_y, loss} per row of FP32 logits."""
    _contig(logits, target, stats)
    M, V = logits.shape
    assert tuple(stats.shape) == (M, 4) and target.shape[0] == M
    _check(lib().ce_fwd(_ptr(logits), _ptr(target), _ptr(stats), M, V, int(ignore_index),
                        _ptr(status), _stream(stream)), "ce_fwd")
    return stats


def ce_bwd(logits: torch.Tensor, target: torch.Tensor, stats: torch.Tensor,
           grad_loss: torch.Tensor, dlogits: torch.Tensor, ignore_index: int = IGNORE_INDEX,
           status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dlogits = (softmax - onehot) * grad_loss in FP32, stored FP32 or BF16.
    grad_loss: one element (broadcast to every row) or M elements."""
    _contig(logits, target, stats, grad_loss, dlogits)
    M, V = logits.shape
    assert tuple(dlogits.shape) == (M, V)
    stride = 0 if grad_loss.numel() == 1 else 1
    if stride == 1:
        assert grad_loss.numel() == M
    _check(lib().ce_bwd(_ptr(logits), _ptr(target), _ptr(stats), _ptr(grad_loss), stride,
                        _ptr(dlogits), _dtype_code(dlogits.dtype), M, V, int(ignore_index),
                        _ptr(status), _stream(stream)), "ce_bwd")
    return dlogits


def lmhead_fwd_ce_workspace_bytes(M: int, V: int) -> int:
    """Scratch bytes lmhead_fwd_ce needs for M tokens and a vocabulary of V."""
    return int(lib().lmhead_fwd_ce_workspace_bytes(int(M), int(V)))


def lmhead_fwd_ce(X: torch.Tensor, W: torch.Tensor, target: torch.Tensor, logits: torch.Tensor,
                  stats: torch.Tensor, workspace: torch.Tensor,
                  ignore_index: int = IGNORE_INDEX, status: Optional[torch.Tensor] = None,
                  stream=None):
    """FP32 logits = X . W^T and stats[M,4] = {m, d, x_y, loss} in one pass over
    the logits; `workspace` is caller-owned scratch (uint8, see
    lmhead_fwd_ce_workspace_bytes)."""
    _contig(X, W, target, logits, stats, workspace)
    M, K = X.shape
    V = W.shape[0]
    assert W.shape[1] == K and tuple(logits.shape) == (M, V) and tuple(stats.shape) == (M, 4)
    assert logits.dtype == torch.float32
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().lmhead_fwd_ce(_ptr(X), _ptr(W), _ptr(target), _ptr(logits), _ptr(stats),
                               _ptr(workspace), nbytes, M, K, V, int(ignore_index), _ptr(status),
                               _stream(stream)), "lmhead_fwd_ce")
    return logits, stats


def lmhead_fwd_ce_noalloc(X: torch.Tensor, W: torch.Tensor, target: torch.Tensor,
                          logits: torch.Tensor, stats: torch.Tensor,
                          ignore_index: int = IGNORE_INDEX, status: Optional[torch.Tensor] = None,
                          stream=None):
    """lmhead_fwd_ce without a workspace, for callers that cannot allocate
    device memory: the partial statistics live in a fixed 8 MiB array inside
    the library (M * 2 * ceil(V/256) <= 1048576).  Calls that overlap on the
    GPU share that array and race."""
    _contig(X, W, target, logits, stats)
    M, K = X.shape
    V = W.shape[0]
    assert W.shape[1] == K and tuple(logits.shape) == (M, V) and tuple(stats.shape) == (M, 4)
    assert logits.dtype == torch.float32
    _check(lib().lmhead_fwd_ce_noalloc(_ptr(X), _ptr(W), _ptr(target), _ptr(logits), _ptr(stats),
                                       M, K, V, int(ignore_index), _ptr(status), _stream(stream)),
           "lmhead_fwd_ce_noalloc")
    return logits, stats


def lmhead_bwd_dx(dlogits: torch.Tensor, W: torch.Tensor, dX: torch.Tensor,
                  status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX[M,K] = dlogits[M,V] . W[V,K]."""
    _contig(dlogits, W, dX)
    M, V = dlogits.shape
    K = W.shape[1]
    assert W.shape[0] == V and tuple(dX.shape) == (M, K)
    _check(lib().lmhead_bwd_dx(_ptr(dlogits), _ptr(W), _ptr(dX), _dtype_code(dX.dtype),
                               M, K, V, _ptr(status), _stream(stream)), "lmhead_bwd_dx")
    return dX


def lmhead_bwd_dw(dlogits: torch.Tensor, X: torch.Tensor, dW: torch.Tensor,
                  status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dW[V,K] = dlogits[M,V]^T . X[M,K]."""
    _contig(dlogits, X, dW)
    M, V = dlogits.shape
    K = X.shape[1]
    assert X.shape[0] == M and tuple(dW.shape) == (V, K)
    _check(lib().lmhead_bwd_dw(_ptr(dlogits), _ptr(X), _ptr(dW), _dtype_code(dW.dtype),
                               M, K, V, _ptr(status), _stream(stream)), "lmhead_bwd_dw")
    return dW


def watchdog_selftest(status: torch.Tensor, limit_us: int = 1000, stream=None) -> None:
    """Make one bounded pipeline wait run out on purpose; sets DEV_PIPE_TIMEOUT."""
    _check(lib().lmh_watchdog_selftest(_ptr(status), int(limit_us), _stream(stream)),
           "lmh_watchdog_selftest")


def gemm_watchdog_selftest(X: torch.Tensor, W: torch.Tensor, logits: torch.Tensor,
                           status: torch.Tensor, limit_ns: int = 1, stream=None) -> None:
    """lmhead_fwd (FP32 logits) with every pipeline wait limited to limit_ns:
    the GEMM's own timeout path, which sets DEV_PIPE_TIMEOUT."""
    _contig(X, W, logits)
    M, K = X.shape
    V = W.shape[0]
    assert W.shape[1] == K and tuple(logits.shape) == (M, V) and logits.dtype == torch.float32
    _check(lib().lmh_gemm_watchdog_selftest(_ptr(X), _ptr(W), _ptr(logits), M, K, V,
                                            int(limit_ns), _ptr(status), _stream(stream)),
           "lmh_gemm_watchdog_selftest")


def lmhead_bwd_dw_acc(dlogits: torch.Tensor, X: torch.Tensor, dW: torch.Tensor,
                      status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dW[V,K] (FP32) += dlogits[M,V]^T . X[M,K]."""
    _contig(dlogits, X, dW)
    M, V = dlogits.shape
    K = X.shape[1]
    assert X.shape[0] == M and tuple(dW.shape) == (V, K) and dW.dtype == torch.float32
    _check(lib().lmhead_bwd_dw_acc(_ptr(dlogits), _ptr(X), _ptr(dW), M, K, V, _ptr(status),
                                   _stream(stream)), "lmhead_bwd_dw_acc")
    return dW


def ce_fwd_shard(logits: torch.Tensor, target: torch.Tensor, shard_stats: torch.Tensor,
                 vocab_offset: int, vocab_total: int, ignore_index: int = IGNORE_INDEX,
                 status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """shard_stats[M,4] = {m_r, d_r, x_y or 0, owner flag} of one vocabulary shard."""
    _contig(logits, target, shard_stats)
    M, V = logits.shape
    assert tuple(shard_stats.shape) == (M, 4)
    _check(lib().ce_fwd_shard(_ptr(logits), _ptr(target), _ptr(shard_stats), M, V,
                              int(vocab_offset), int(vocab_total), int(ignore_index),
                              _ptr(status), _stream(stream)), "ce_fwd_shard")
    return shard_stats


def ce_merge_shards(shard_stats: torch.Tensor, target: torch.Tensor, stats: torch.Tensor,
                    vocab_total: int, ignore_index: int = IGNORE_INDEX,
                    status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """stats[M,4] = {m, d, x_y, loss} from shard_stats[R,M,4] (shard-major)."""
    _contig(shard_stats, target, stats)
    R, M, four = shard_stats.shape
    assert four == 4 and tuple(stats.shape) == (M, 4)
    _check(lib().ce_merge_shards(_ptr(shard_stats), R, _ptr(target), _ptr(stats), M,
                                 int(vocab_total), int(ignore_index), _ptr(status),
                                 _stream(stream)), "ce_merge_shards")
    return stats


def ce_bwd_shard(logits: torch.Tensor, target: torch.Tensor, stats: torch.Tensor,
                 grad_loss: torch.Tensor, dlogits: torch.Tensor, vocab_offset: int,
                 vocab_total: int, ignore_index: int = IGNORE_INDEX,
                 status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ce_bwd on one vocabulary shard with the merged statistics."""
    _contig(logits, target, stats, grad_loss, dlogits)
    M, V = logits.shape
    stride = 0 if grad_loss.numel() == 1 else 1
    _check(lib().ce_bwd_shard(_ptr(logits), _ptr(target), _ptr(stats), _ptr(grad_loss), stride,
                              _ptr(dlogits), _dtype_code(dlogits.dtype), M, V, int(vocab_offset),
                              int(vocab_total), int(ignore_index), _ptr(status), _stream(stream)),
           "ce_bwd_shard")
    return dlogits


_F32, _B16, _I32, _I64 = ((d,) for d in (torch.float32, torch.bfloat16, torch.int32, torch.int64))
_LOGITS = _F32 + _B16


def _refuse(name: str, t: torch.Tensor, shape, dtypes, dev: int):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    raise ValueError(f"{name} is on another device than the call's first tensor")


def _take(dev: int, *args):
    """The addresses of a call's tensors, each given as (name, tensor, shape, dtypes)
    and checked: contiguous, on device number `dev`.  None stays None."""
    out = []
    for name, t, shape, dtypes in args:
        if t is None:
            out.append(None)
            continue
        if t.shape != shape or t.dtype not in dtypes or not t.is_contiguous() or t.get_device() != dev:
            _refuse(name, t, shape, dtypes, dev)
        out.append(t.data_ptr())
    return out


def _workspace(t: torch.Tensor, dev: int):
    """(address, bytes) of a caller's scratch buffer."""
    if not t.is_contiguous() or t.get_device() != dev:
        raise ValueError("workspace must be contiguous and on the device of the call's first tensor")
    return t.data_ptr(), t.numel() * t.element_size()


def _on(dev: int, stream, fn, *args) -> int:
    """fn(*args, stream) with device number `dev` current; stream None is that
    device's current stream."""
    if dev < 0:
        raise ValueError("expected CUDA tensors (the library has no CPU path)")
    # the raw handle, without the Stream object around it (1.5 us less per call)
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch.cuda.current_device():
        return fn(*args, s)
    with torch.cuda.device(dev):
        return fn(*args, s)


def beam_select_workspace_bytes(N: int, W: int, V: int, C: int) -> int:
    """Scratch bytes beam_select needs for N entries of W beams, a vocabulary of
    V and C candidates (-1 for sizes out of range)."""
    return int(lib().beam_select_workspace_bytes(int(N), int(W), int(V), int(C)))


def beam_select(logits: torch.Tensor, scores: torch.Tensor, cand_score: torch.Tensor,
                cand_beam: torch.Tensor, cand_token: torch.Tensor,
                next_score: Optional[torch.Tensor], next_beam: Optional[torch.Tensor],
                next_token: Optional[torch.Tensor], workspace: torch.Tensor, eos: int = -1,
                done: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                stream=None):
    """One step of beam search: the C best continuations of logits[N,W,V] (FP32 or
    BF16) with beam scores[N,W] into cand_*[N,C] (score FP32, beam int32, token
    int64; best first, ties to the lower beam and token), and the first W whose
    token is not `eos` into next_*[N,W] (all three None to skip).  Entries with
    done[n] != 0 (int32) are not read and keep their beams."""
    if logits.dim() != 3 or cand_score.dim() != 2:
        raise ValueError("expected logits [N,W,V] and cand_score [N,C]")
    N, W, V = logits.shape
    nw, nc, dev = (N, W), (N, cand_score.shape[1]), logits.get_device()
    wp, wn = _workspace(workspace, dev)
    lg, *ptrs, st = _take(
        dev, ("logits", logits, (N, W, V), _LOGITS), ("scores", scores, nw, _F32),
        ("done", done, (N,), _I32), ("cand_score", cand_score, nc, _F32),
        ("cand_beam", cand_beam, nc, _I32), ("cand_token", cand_token, nc, _I64),
        ("next_score", next_score, nw, _F32), ("next_beam", next_beam, nw, _I32),
        ("next_token", next_token, nw, _I64), ("status", status, (1,), _I32))
    code = _on(dev, stream, lib().beam_select, lg, F32 if logits.dtype is torch.float32 else BF16,
               *ptrs, wp, wn, N, W, V, nc[1], int(eos), st)
    if code:
        raise LmhError(code, "beam_select")
    return cand_score, cand_beam, cand_token, next_score, next_beam, next_token


@functools.lru_cache(maxsize=256)
def _state_geometry(shape, strides, es: int, entry_dim: int):
    """(run_bytes, outer extents, outer strides) of a state seen as elements
    [.., n, w, ..]: the dimensions that are contiguous below every other one form
    the run, the others are merged where one steps over the next."""
    dims = sorted((strides[d] * es, shape[d]) for d in range(len(shape))
                  if d not in (entry_dim, entry_dim + 1) and shape[d] != 1)
    run = es
    while dims and dims[0][0] == run:
        run *= dims.pop(0)[1]
    merged = []
    for st, n in dims:
        if merged and st == merged[-1][0] * merged[-1][1]:
            merged[-1] = (merged[-1][0], merged[-1][1] * n)
        else:
            merged.append((st, n))
    if len(merged) > 3:
        raise ValueError("a state may have at most three strided dimensions beside its beams")
    k = len(merged)
    return run, (ctypes.c_int64 * k)(*[n for _, n in merged]), (ctypes.c_int64 * k)(*[st for st, _ in merged])


def beam_reorder(states, parents: torch.Tensor, entry_dim: int = 0,
                 status: Optional[torch.Tensor] = None, stream=None):
    """Each state (one tensor or a list, all of one shape and strides, any dtype) is
    put in the order of its beams' parents, in place: state[.., n, w, ..] becomes the
    old state[.., n, parents[n, w], ..], with n in dimension entry_dim and w in the
    next.  parents: [N, W] int32, as beam_select's next_beam.  Strided views (the
    filled part of a cache) are taken as they are.  States that share memory are
    refused (among each 128 of the list, one launch's worth)."""
    states = [states] if isinstance(states, torch.Tensor) else list(states)
    if parents.dim() != 2 or not states:
        raise ValueError("expected parents [N,W] and at least one state")
    (N, W), dev = parents.shape, parents.get_device()
    first = states[0]
    shape, strides, dtype, es = tuple(first.shape), first.stride(), first.dtype, first.element_size()
    if not 0 <= entry_dim <= len(shape) - 2 or shape[entry_dim:entry_dim + 2] != (N, W):
        raise ValueError(f"dimensions {entry_dim} and {entry_dim + 1} of a state must be {(N, W)}")
    for t in states:
        if t.shape != shape or t.stride() != strides or t.dtype is not dtype:
            raise ValueError("the states of one call must have one shape, dtype and strides")
        if t.get_device() != dev:
            raise ValueError("the states and parents must be on one device")
    pp, sp = _take(dev, ("parents", parents, (N, W), _I32), ("status", status, (1,), _I32))
    if 0 in shape:
        return states
    run, outer, outer_strides = _state_geometry(shape, strides, es, entry_dim)
    addresses = [t.data_ptr() for t in states]
    if len(set(addresses)) < len(addresses):
        raise ValueError("a state is given twice")
    for i in range(0, len(states), 128):
        part = addresses[i:i + 128]
        ptrs = (ctypes.c_void_p * len(part))(*part)
        code = _on(dev, stream, lib().beam_reorder, ptrs, len(part), pp, N, W, strides[entry_dim] * es,
                   strides[entry_dim + 1] * es, run, outer, outer_strides, len(outer), sp)
        if code:
            raise LmhError(code, "beam_reorder")
    return states


def lmhead_lora_workspace_bytes(M: int, K: int, V: int, R: int, N: int) -> int:
    """Scratch bytes each of the adapter calls needs at most for M tokens and N
    adapters of rank R (-1 for sizes out of range)."""
    return int(lib().lmhead_lora_workspace_bytes(int(M), int(K), int(V), int(R), int(N)))


def lmhead_fwd_lora(X: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                    scale: torch.Tensor, adapter: torch.Tensor, u: torch.Tensor,
                    logits: torch.Tensor, workspace: torch.Tensor,
                    status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """logits[M,V] (FP32 or BF16) = X[M,K] . W[V,K]^T + u . B_a^T with
    u[M,R] (FP32, written) = scale[a] X . A_a^T, the adapter a = adapter[i] (int32,
    -1 for none) of each token out of A[N,R,K], B[N,V,R] (BF16), scale[N] (FP32)."""
    if X.dim() != 2 or W.dim() != 2 or A.dim() != 3:
        raise ValueError("expected X [M,K], W [V,K], A [N,R,K]")
    (M, K), V, (N, R) = X.shape, W.shape[0], A.shape[:2]
    dev = X.get_device()
    wp, wn = _workspace(workspace, dev)
    *ptrs, st = _take(dev, ("X", X, (M, K), _B16), ("W", W, (V, K), _B16), ("A", A, (N, R, K), _B16),
                      ("B", B, (N, V, R), _B16), ("scale", scale, (N,), _F32),
                      ("adapter", adapter, (M,), _I32), ("u", u, (M, R), _F32),
                      ("logits", logits, (M, V), _LOGITS), ("status", status, (1,), _I32))
    code = _on(dev, stream, lib().lmhead_fwd_lora, *ptrs,
               F32 if logits.dtype is torch.float32 else BF16, wp, wn, M, K, V, R, N, st)
    if code:
        raise LmhError(code, "lmhead_fwd_lora")
    return logits


def lmhead_bwd_dx_lora(dlogits: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                       scale: torch.Tensor, adapter: torch.Tensor, g: torch.Tensor,
                       dX: torch.Tensor, workspace: torch.Tensor,
                       status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX[M,K] (FP32 or BF16) = dlogits[M,V] . W + g . A_a with g[M,R] (FP32, written)
    = scale[a] dlogits . B_a: the input gradient of lmhead_fwd_lora."""
    if dlogits.dim() != 2 or W.dim() != 2 or A.dim() != 3:
        raise ValueError("expected dlogits [M,V], W [V,K], A [N,R,K]")
    (M, V), K, (N, R) = dlogits.shape, W.shape[1], A.shape[:2]
    dev = dlogits.get_device()
    wp, wn = _workspace(workspace, dev)
    *ptrs, st = _take(dev, ("dlogits", dlogits, (M, V), _B16), ("W", W, (V, K), _B16),
                      ("A", A, (N, R, K), _B16), ("B", B, (N, V, R), _B16), ("scale", scale, (N,), _F32),
                      ("adapter", adapter, (M,), _I32), ("g", g, (M, R), _F32),
                      ("dX", dX, (M, K), _LOGITS), ("status", status, (1,), _I32))
    code = _on(dev, stream, lib().lmhead_bwd_dx_lora, *ptrs,
               F32 if dX.dtype is torch.float32 else BF16, wp, wn, M, K, V, R, N, st)
    if code:
        raise LmhError(code, "lmhead_bwd_dx_lora")
    return dX


def lmhead_bwd_lora(dlogits: torch.Tensor, X: torch.Tensor, u: torch.Tensor, g: torch.Tensor,
                    adapter: torch.Tensor, dA: torch.Tensor, dB: torch.Tensor,
                    workspace: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None):
    """The adapters' gradients dA[N,R,K], dB[N,V,R] (FP32) from the u of
    lmhead_fwd_lora and the g of lmhead_bwd_dx_lora: over the tokens of each adapter,
    dA_a = g^T . X and dB_a = dlogits^T . u (zeros for an adapter without tokens)."""
    if dlogits.dim() != 2 or X.dim() != 2 or dA.dim() != 3:
        raise ValueError("expected dlogits [M,V], X [M,K], dA [N,R,K]")
    (M, V), K, (N, R) = dlogits.shape, X.shape[1], dA.shape[:2]
    dev = dlogits.get_device()
    wp, wn = _workspace(workspace, dev)
    *ptrs, st = _take(dev, ("dlogits", dlogits, (M, V), _B16), ("X", X, (M, K), _B16),
                      ("u", u, (M, R), _F32), ("g", g, (M, R), _F32), ("adapter", adapter, (M,), _I32),
                      ("dA", dA, (N, R, K), _F32), ("dB", dB, (N, V, R), _F32),
                      ("status", status, (1,), _I32))
    code = _on(dev, stream, lib().lmhead_bwd_lora, *ptrs, wp, wn, M, K, V, R, N, st)
    if code:
        raise LmhError(code, "lmhead_bwd_lora")
    return dA, dB
