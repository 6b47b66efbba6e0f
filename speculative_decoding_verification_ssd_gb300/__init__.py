"""Python binding of libssd: batched speculative-decoding verification and the
Saguaro speculation-cache kernels for GB300 (sm_103a).

The functions here carry the names of the C ABI in ``include/ssd.h`` and only
marshal arguments: torch tensors provide device memory and the CUDA stream,
every step of the computation runs in libssd's kernels.  If ``libssd.so`` has
not been built (``__graft_entry__.build()`` or ``python -m
speculative_decoding_verification_ssd_gb300._build``), every call raises:
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os

import numpy as np
import torch

from . import _build

SSD_OK = 0
SSD_ERR_INVALID_ARG = 1
SSD_ERR_DTYPE = 2
SSD_ERR_CUDA = 3
SSD_ERR_WORKSPACE = 4
SSD_ERR_UNSUPPORTED = 5

SSD_F32 = 0
SSD_BF16 = 1
SSD_F16 = 2

SSD_DEV_BAD_TOKEN = 1
SSD_DEV_BAD_TEMPERATURE = 2
SSD_DEV_NONFINITE = 4
SSD_DEV_TIMEOUT = 8
SSD_DEV_BAD_PAGE = 16
SSD_DEV_NO_PAGES = 32
SSD_DEV_BAD_LENGTH = 64
SSD_DEV_BAD_PARAM = 128
SSD_DEV_LOW_LOGITS = 256
SSD_DEV_BAD_TREE = 512

SSD_MAX_K = 32
SSD_MAX_F = 256
SSD_KV_MAX_B = 4096
SSD_TREE_MAX = 1024
SSD_DROPPED_LOGIT = -1e5

LIB_PATH = _build.LIB

# Symbols declared in include/ssd.h.
ABI_SYMBOLS = ("ssd_strerror", "ssd_version", "ssd_workspace_size", "ssd_verify", "ssd_fanout",
               "ssd_reshape_draft", "ssd_build_cache", "ssd_cache_lookup", "ssd_round",
               "ssd_noalloc_max_scratch", "ssd_round_noalloc", "ssd_fanout_uniform",
               "ssd_backup_fill", "ssd_draft_cache", "ssd_verify_sigma", "ssd_round_sigma",
               "ssd_set_dispatch", "ssd_check_wait_timeout", "ssd_verify_ld", "ssd_round_ld",
               "ssd_host_staging_size", "ssd_round_host", "ssd_last_kernel", "ssd_workspace_size_v",
               "ssd_kv_plan", "ssd_kv_append", "ssd_kv_workspace_size", "ssd_kv_attend", "ssd_sample",
               "ssd_qk_rope", "ssd_tree_plan", "ssd_kv_tree_workspace_size", "ssd_kv_attend_tree", "ssd_tree_accept",
               "ssd_kv_compact", "ssd_check_tree_timeout")


class SSDError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libssd (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libssd is not built ({LIB_PATH} missing); run "
                               "`python -m speculative_decoding_verification_ssd_gb300._build`")
        L = ctypes.CDLL(LIB_PATH)
        P, i, d, z = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_size_t
        f = ctypes.c_float
        L.ssd_strerror.argtypes = [i]
        L.ssd_strerror.restype = ctypes.c_char_p
        L.ssd_version.argtypes = []
        L.ssd_version.restype = ctypes.c_char_p
        L.ssd_last_kernel.argtypes = []
        L.ssd_last_kernel.restype = ctypes.c_char_p
        L.ssd_workspace_size.argtypes = [i, i]
        L.ssd_workspace_size.restype = z
        L.ssd_workspace_size_v.argtypes = [i, i, i, i, i]
        L.ssd_workspace_size_v.restype = z
        L.ssd_verify.argtypes = [P, P, i, i, i, i, i, P, P, P, P, P, P, P, P, P, z, P, P]
        L.ssd_verify.restype = i
        L.ssd_fanout.argtypes = [i, i, d, d, i, P, P]
        L.ssd_fanout.restype = i
        L.ssd_reshape_draft.argtypes = [P, i, i, i, P, i, f, P, P, P, P]
        L.ssd_reshape_draft.restype = i
        L.ssd_build_cache.argtypes = [P, P, i, i, i, i, i, P, P, P, P, i, P, P, z, P, P]
        L.ssd_build_cache.restype = i
        L.ssd_cache_lookup.argtypes = [P, i, i, i, P, P, P, P, P, P]
        L.ssd_cache_lookup.restype = i
        L.ssd_round.argtypes = [P, P, i, i, i, i, i, P, P, P, P, P, i, P, P, P, P, P, P, P, P, z,
                                P, P]
        L.ssd_round.restype = i
        L.ssd_noalloc_max_scratch.argtypes = []
        L.ssd_noalloc_max_scratch.restype = z
        L.ssd_round_noalloc.argtypes = [P, P, i, i, i, i, i, P, P, P, P, P, i, P, P, P, P, P, P, P, P,
                                        P]
        L.ssd_round_noalloc.restype = i
        L.ssd_fanout_uniform.argtypes = [i, i, i, P, P]
        L.ssd_fanout_uniform.restype = i
        L.ssd_backup_fill.argtypes = [P, P, i, i, i, P, P]
        L.ssd_backup_fill.restype = i
        L.ssd_draft_cache.argtypes = [P, i, i, i, i, P, P, i, f, P, P, P, P]
        L.ssd_draft_cache.restype = i
        L.ssd_verify_sigma.argtypes = [P, P, i, i, i, i, i, P, P, P, P, f, P, P, P, P, P, P, z, P, P]
        L.ssd_verify_sigma.restype = i
        L.ssd_round_sigma.argtypes = [P, P, i, i, i, i, i, P, P, P, P, f, P, P, i, P, P, P, P, P, P,
                                      P, P, z, P, P]
        L.ssd_round_sigma.restype = i
        L.ssd_set_dispatch.argtypes = [i]
        L.ssd_set_dispatch.restype = i
        L.ssd_check_wait_timeout.argtypes = [P, i, P]
        L.ssd_check_wait_timeout.restype = i
        L.ssd_verify_ld.argtypes = [P, P, i, i, i, i, i, i, P, P, P, P, P, P, P, P, P, z, P, P]
        L.ssd_verify_ld.restype = i
        L.ssd_round_ld.argtypes = [P, P, i, i, i, i, i, i, P, P, P, P, P, i, P, P, P, P, P, P, P, P,
                                   z, P, P]
        L.ssd_round_ld.restype = i
        L.ssd_host_staging_size.argtypes = [i, i, i, i, i]
        L.ssd_host_staging_size.restype = z
        L.ssd_round_host.argtypes = [P, P, i, i, i, i, P, P, P, P, i, P, P, P, P, P, P, z, P, z, P, P,
                                     P]
        L.ssd_round_host.restype = i
        n = ctypes.c_int64
        L.ssd_kv_plan.argtypes = [P, P, P, P, i, P, i, P, P, i, i, i, P, P, P, P, P, P]
        L.ssd_kv_plan.restype = i
        L.ssd_kv_append.argtypes = [P, P, i, n, n, P, i, i, i, P, P, P, P, i, i, P, P]
        L.ssd_kv_append.restype = i
        L.ssd_kv_workspace_size.argtypes = []
        L.ssd_kv_workspace_size.restype = z
        L.ssd_kv_attend.argtypes = [P, i, n, P, P, P, P, i, i, i, i, i, P, i, P, P, i, i, i, f, i, P, P, z,
                                    P, P]
        L.ssd_kv_attend.restype = i
        L.ssd_sample.argtypes = [P, i, i, i, n, P, P, P, P, P, P, P, P, P, P]
        L.ssd_sample.restype = i
        L.ssd_qk_rope.argtypes = [P, P, i, n, n, i, i, i, i, P, P, f, P, P, i, i, P, P, n, n, P]
        L.ssd_qk_rope.restype = i
        L.ssd_tree_plan.argtypes = [P, P, P, i, i, i, P, P, P, P]
        L.ssd_tree_plan.restype = i
        L.ssd_kv_tree_workspace_size.argtypes = []
        L.ssd_kv_tree_workspace_size.restype = z
        L.ssd_kv_attend_tree.argtypes = [P, i, n, P, P, P, P, i, i, i, i, i, P, i, P, P, P, i, i, i, f, i, P, P, z, P, P]
        L.ssd_kv_attend_tree.restype = i
        L.ssd_check_tree_timeout.argtypes = [i] + L.ssd_kv_attend_tree.argtypes
        L.ssd_check_tree_timeout.restype = i
        L.ssd_tree_accept.argtypes = [P, P, P, P, i, i, i, i, P, P, P, P, P]
        L.ssd_tree_accept.restype = i
        L.ssd_kv_compact.argtypes = [P, P, P, i, i, P, i, i, i, P, P, P, P, i, i, P, P]
        L.ssd_kv_compact.restype = i
        _lib = L
    return _lib


SSD_DISPATCH_AUTO, SSD_DISPATCH_STREAM, SSD_DISPATCH_CLUSTER, SSD_DISPATCH_SLICE, SSD_DISPATCH_WIDE = 0, 1, 2, 3, 4


def ssd_set_dispatch(policy: int) -> int:
    """Kernel choice for aligned rows (process-wide); returns the previous policy."""
    prev = int(lib().ssd_set_dispatch(int(policy)))
    if prev < 0:
        raise ValueError(f"unknown dispatch policy {policy}")
    return prev


def ssd_check_wait_timeout(dev_status, limit_ms: int, *, stream=None):
    """Runs the bounded-wait check: a wait nothing completes gives up after limit_ms
    and ORs SSD_DEV_TIMEOUT into dev_status (a device int32 tensor)."""
    _dev(dev_status, "dev_status", torch.int32)
    _check(lib().ssd_check_wait_timeout(_ptr(dev_status), int(limit_ms), _stream(stream)),
           "ssd_check_wait_timeout")
    return dev_status


def strerror(status: int) -> str:
    try:
        return lib().ssd_strerror(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def ssd_last_kernel() -> str:
    """The kernel the calling thread's last verify / cache / round call launched."""
    return lib().ssd_last_kernel().decode()


def version() -> str:
    return lib().ssd_version().decode()


def _check(status: int, where: str):
    if status != SSD_OK:
        raise SSDError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data_as(ctypes.c_void_p)
    return ctypes.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _logit_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SSD_F32
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


# ---------------------------------------------------------------------------
# Host-only calls.
# ---------------------------------------------------------------------------

def ssd_workspace_size(B: int, K: int) -> int:
    return int(lib().ssd_workspace_size(int(B), int(K)))


def ssd_workspace_size_v(B: int, K: int, V: int, dtype: int, budget: int = 0) -> int:
    return int(lib().ssd_workspace_size_v(int(B), int(K), int(V), int(dtype), int(budget)))


def ssd_fanout(K: int, budget: int, a_p: float, r: float, V: int):
    """Geometric fan-out: (F [K+1], off [K+2]) as numpy int32 arrays."""
    F = np.empty(K + 1, np.int32)
    off = np.empty(K + 2, np.int32)
    _check(lib().ssd_fanout(int(K), int(budget), float(a_p), float(r), int(V), _ptr(F), _ptr(off)),
           "ssd_fanout")
    return F, off


def ssd_fanout_uniform(K: int, budget: int, V: int):
    """Uniform fan-out: (F [K+1], off [K+2]) as numpy int32 arrays."""
    F = np.empty(K + 1, np.int32)
    off = np.empty(K + 2, np.int32)
    _check(lib().ssd_fanout_uniform(int(K), int(budget), int(V), _ptr(F), _ptr(off)),
           "ssd_fanout_uniform")
    return F, off


def workspace(B: int, K: int, device=None, V: int | None = None, dtype: int | None = None,
              budget: int = 0) -> torch.Tensor:
    """A zero-filled workspace for B sequences of K drafted tokens; with V and dtype
    (and the cache budget) it also holds the slice kernel's regions."""
    if V is not None and dtype is not None:
        n = ssd_workspace_size_v(B, K, V, dtype, budget)
    else:
        n = ssd_workspace_size(B, K)
    if n == 0:
        raise ValueError("invalid workspace arguments")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _workspace(ws, B, K, device, V=None, dtype=None, budget=0):
    if ws is None:
        ws = workspace(B, K, device, V, dtype, budget)
    _dev(ws, "workspace", torch.uint8)
    return ws


def _row_stride(t, name):
    """Elements between consecutive rows of a [B, R, V] logit tensor whose rows are
    contiguous and evenly spaced (a contiguous tensor, or a [..., :V] view of one
    with a longer row); raises for any other layout."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [B, rows, V]")
    B, R, V = t.shape
    ld = t.stride(1) if R > 1 else (t.stride(0) if B > 1 else V)
    if t.stride(2) != 1 or ld < V or (R > 1 and B > 1 and t.stride(0) != R * ld):
        raise ValueError(f"{name} rows must be contiguous and evenly spaced")
    return int(ld)


def _shapes(tgt, drf, tokens, allow_ld=False):
    if tgt.dim() != 3 or drf.dim() != 3:
        raise ValueError("tgt must be [B, K+1, V] and drf [B, K or K+1, V]")
    if allow_ld:
        ld_t, ld_d = _row_stride(tgt, "tgt"), _row_stride(drf, "drf")
        if tgt.shape[1] == 1 and tgt.shape[0] == 1:
            ld_t = ld_d
        if drf.shape[1] == 1 and drf.shape[0] == 1:
            ld_d = ld_t
        if ld_t != ld_d:
            raise ValueError("tgt and drf must share one row stride")
    else:
        _dev(tgt, "tgt")
        _dev(drf, "drf")
        ld_t = int(tgt.shape[2])
    B, K1, V = tgt.shape
    K = K1 - 1
    if drf.shape[0] != B or drf.shape[2] != V or drf.dtype != tgt.dtype:
        raise ValueError("drf must match tgt in batch, vocabulary and dtype")
    _dev(tokens, "tokens", torch.int32)
    if tuple(tokens.shape) != (B, K):
        raise ValueError("tokens must be [B, K]")
    if allow_ld:
        return B, K, V, int(drf.shape[1]), ld_t
    return B, K, V, int(drf.shape[1])


def _opt(t, name, dtype):
    return None if t is None else _dev(t, name, dtype)


def _F_host(F):
    return np.ascontiguousarray(np.asarray(F, dtype=np.int32))


# ---------------------------------------------------------------------------
# Device calls.
# ---------------------------------------------------------------------------

def ssd_verify(tgt, drf, tokens, uniforms, temperature, reshape=None, *, accept_len=None,
               bonus=None, p_tok=None, q_tok=None, probs=True, workspace=None, dev_status=None,
               stream=None):
    """Verify one batch: returns dict(accept_len, bonus[, p_tok, q_tok]).  The logit
    tensors may be [..., :V] views of rows with a longer stride (same for both)."""
    B, K, V, drf_rows, ld = _shapes(tgt, drf, tokens, allow_ld=True)
    dev = tgt.device
    _dev(uniforms, "uniforms", torch.float32)
    _dev(temperature, "temperature", torch.float32)
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    bonus = bonus if bonus is not None else torch.empty(B, dtype=torch.int32, device=dev)
    if probs:
        p_tok = p_tok if p_tok is not None else torch.empty((B, K), dtype=torch.float32, device=dev)
        q_tok = q_tok if q_tok is not None else torch.empty((B, K), dtype=torch.float32, device=dev)
    ws = _workspace(workspace, B, K, dev, V, _logit_dtype(tgt))
    _opt(reshape, "reshape", torch.int32)
    _check(lib().ssd_verify_ld(
        _ptr(tgt), _ptr(drf), _logit_dtype(tgt), B, K, V, ld, drf_rows, _ptr(tokens), _ptr(uniforms),
        _ptr(temperature), _ptr(reshape), _ptr(accept_len), _ptr(bonus), _ptr(p_tok), _ptr(q_tok),
        _ptr(ws), ws.numel(), _ptr(_opt(dev_status, "dev_status", torch.int32)), _stream(stream)),
        "ssd_verify_ld")
    out = {"accept_len": accept_len, "bonus": bonus}
    if probs:
        out.update(p_tok=p_tok, q_tok=q_tok)
    return out


def ssd_build_cache(tgt, drf, tokens, temperature, F, budget, reshape=None, *, cache_tok=None,
                    workspace=None, dev_status=None, stream=None):
    """Speculation-cache keys: cache_tok [B, budget] int32 (segment k = top-F_k)."""
    B, K, V, drf_rows = _shapes(tgt, drf, tokens)
    dev = tgt.device
    _dev(temperature, "temperature", torch.float32)
    Fh = _F_host(F)
    cache_tok = cache_tok if cache_tok is not None else torch.full((B, budget), -1, dtype=torch.int32, device=dev)
    ws = _workspace(workspace, B, K, dev, V, _logit_dtype(tgt), int(budget))
    _check(lib().ssd_build_cache(
        _ptr(tgt), _ptr(drf), _logit_dtype(tgt), B, K, V, drf_rows, _ptr(tokens),
        _ptr(temperature), _ptr(_opt(reshape, "reshape", torch.int32)), _ptr(Fh), int(budget),
        _ptr(cache_tok), _ptr(ws), ws.numel(), _ptr(_opt(dev_status, "dev_status", torch.int32)),
        _stream(stream)), "ssd_build_cache")
    return cache_tok


def ssd_cache_lookup(cache_tok, F, accept_len, bonus, *, hit=None, slot=None, stream=None):
    """Hit test of the true outcome (a, t*): (hit [B] uint8, slot [B] int32)."""
    _dev(cache_tok, "cache_tok", torch.int32)
    B, budget = cache_tok.shape
    Fh = _F_host(F)
    K = len(Fh) - 1
    dev = cache_tok.device
    hit = hit if hit is not None else torch.empty(B, dtype=torch.uint8, device=dev)
    slot = slot if slot is not None else torch.empty(B, dtype=torch.int32, device=dev)
    _check(lib().ssd_cache_lookup(
        _ptr(cache_tok), B, K, budget, _ptr(Fh), _ptr(_dev(accept_len, "accept_len", torch.int32)),
        _ptr(_dev(bonus, "bonus", torch.int32)), _ptr(hit), _ptr(slot), _stream(stream)),
        "ssd_cache_lookup")
    return hit, slot


def ssd_backup_fill(hit, uniforms, V: int, next_tokens, *, stream=None):
    """Random-token backup for the sequences that missed: next_tokens [B, K] int32 is
    written in place where hit[b] == 0 (token floor(u * V)); returns next_tokens."""
    _dev(hit, "hit", torch.uint8)
    _dev(uniforms, "uniforms", torch.float32)
    _dev(next_tokens, "next_tokens", torch.int32)
    if uniforms.dim() != 2 or tuple(next_tokens.shape) != tuple(uniforms.shape) \
            or hit.shape != (uniforms.shape[0],):
        raise ValueError("uniforms and next_tokens must be [B, K] and hit [B]")
    B, K = uniforms.shape
    _check(lib().ssd_backup_fill(_ptr(hit), _ptr(uniforms), B, K, int(V), _ptr(next_tokens),
                                 _stream(stream)), "ssd_backup_fill")
    return next_tokens


def ssd_round(tgt, drf, tokens, uniforms, temperature, F, budget, reshape=None, *, out=None,
              probs=True, workspace=None, dev_status=None, stream=None):
    """One fused SSD round: verify + cache build + lookup.  Returns a dict of outputs.
    The logit tensors may be [..., :V] views of rows with a longer stride."""
    B, K, V, drf_rows, ld = _shapes(tgt, drf, tokens, allow_ld=True)
    dev = tgt.device
    _dev(uniforms, "uniforms", torch.float32)
    _dev(temperature, "temperature", torch.float32)
    Fh = _F_host(F)
    o = dict(out) if out is not None else {}
    if not probs:
        o.pop("p_tok", None)
        o.pop("q_tok", None)
    # allocate only what the caller did not supply (no work is enqueued otherwise)
    if "accept_len" not in o:
        o["accept_len"] = torch.empty(B, dtype=torch.int32, device=dev)
    if "bonus" not in o:
        o["bonus"] = torch.empty(B, dtype=torch.int32, device=dev)
    if probs and "p_tok" not in o:
        o["p_tok"] = torch.empty((B, K), dtype=torch.float32, device=dev)
    if probs and "q_tok" not in o:
        o["q_tok"] = torch.empty((B, K), dtype=torch.float32, device=dev)
    if "cache_tok" not in o:
        o["cache_tok"] = torch.full((B, budget), -1, dtype=torch.int32, device=dev)
    if "hit" not in o:
        o["hit"] = torch.empty(B, dtype=torch.uint8, device=dev)
    if "slot" not in o:
        o["slot"] = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(workspace, B, K, dev, V, _logit_dtype(tgt), int(budget))
    _check(lib().ssd_round_ld(
        _ptr(tgt), _ptr(drf), _logit_dtype(tgt), B, K, V, ld, drf_rows, _ptr(tokens), _ptr(uniforms),
        _ptr(temperature), _ptr(_opt(reshape, "reshape", torch.int32)), _ptr(Fh), int(budget),
        _ptr(o["accept_len"]), _ptr(o["bonus"]), _ptr(o.get("p_tok")), _ptr(o.get("q_tok")),
        _ptr(o["cache_tok"]), _ptr(o["hit"]), _ptr(o["slot"]), _ptr(ws), ws.numel(),
        _ptr(_opt(dev_status, "dev_status", torch.int32)), _stream(stream)), "ssd_round_ld")
    return o


def _host(t, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise TypeError(f"{name} must be a host (CPU) tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def ssd_host_staging_size(dtype: int, B: int, K: int, V: int, budget: int) -> int:
    """Device bytes ssd_round_host needs for its copies of one round's inputs and outputs."""
    return int(lib().ssd_host_staging_size(int(dtype), int(B), int(K), int(V), int(budget)))


def ssd_round_host(tgt, drf, tokens, uniforms, temperature, F, budget, *, out=None, staging=None,
                   workspace=None, dev_status=None, stream=None, device=None):
    """ssd_round on host tensors (page-locked ones copy asynchronously): the inputs
    are copied to the device (the draft rows of sampled sequences only), the round
    runs and its results are copied back, all on `stream`.  Returns (outputs, h2d):
    a dict of host tensors accept_len, bonus, cache_tok, hit, slot -- valid once the
    stream has completed -- and the bytes copied to the device."""
    _host(tgt, "tgt")
    _host(drf, "drf", tgt.dtype)
    if tgt.dim() != 3 or drf.dim() != 3:
        raise ValueError("tgt must be [B, K+1, V] and drf [B, K, V]")
    B, K1, V = tgt.shape
    K = K1 - 1
    if tuple(drf.shape) != (B, K, V):
        raise ValueError("drf must be [B, K, V]")
    _host(tokens, "tokens", torch.int32)
    _host(uniforms, "uniforms", torch.float32)
    _host(temperature, "temperature", torch.float32)
    if tuple(tokens.shape) != (B, K) or tuple(uniforms.shape) != (B, K + 1) or tuple(temperature.shape) != (B,):
        raise ValueError("tokens [B, K], uniforms [B, K+1] and temperature [B] expected")
    dt = _logit_dtype(tgt)
    Fh = _F_host(F)
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    o = dict(out) if out is not None else {}
    shapes = {"accept_len": ((B,), torch.int32), "bonus": ((B,), torch.int32),
              "cache_tok": ((B, int(budget)), torch.int32), "hit": ((B,), torch.uint8),
              "slot": ((B,), torch.int32)}
    for k, (shp, dty) in shapes.items():
        if k not in o:
            o[k] = torch.empty(shp, dtype=dty).pin_memory()
        _host(o[k], k, dty)
    need = ssd_host_staging_size(dt, B, K, V, budget)
    if need == 0:
        raise ValueError("invalid sizes for ssd_round_host")
    if staging is None:
        staging = torch.empty(need, dtype=torch.uint8, device=dev)
    _dev(staging, "staging", torch.uint8)
    ws = _workspace(workspace, B, K, dev, V, dt, int(budget))
    moved = ctypes.c_size_t(0)
    _check(lib().ssd_round_host(
        _ptr(tgt), _ptr(drf), dt, B, K, V, _ptr(tokens), _ptr(uniforms), _ptr(temperature), _ptr(Fh),
        int(budget), _ptr(o["accept_len"]), _ptr(o["bonus"]), _ptr(o["cache_tok"]), _ptr(o["hit"]),
        _ptr(o["slot"]), _ptr(staging), staging.numel(), _ptr(ws), ws.numel(),
        _ptr(_opt(dev_status, "dev_status", torch.int32)), ctypes.c_void_p(ctypes.addressof(moved)),
        _stream(stream)), "ssd_round_host")
    return o, int(moved.value)


def _sigma_args(sigma_F, K, B, desc_out, dev):
    Fs = _F_host(sigma_F)
    if Fs.shape != (K,):
        raise ValueError("sigma_F must have K entries")
    desc_out = desc_out if desc_out is not None else torch.zeros((B * K, 4), dtype=torch.int32,
                                                                 device=dev)
    _dev(desc_out, "desc_out", torch.int32)
    if desc_out.numel() != B * K * 4:
        raise ValueError("desc_out must hold B*K descriptors")
    return Fs, desc_out


def ssd_verify_sigma(tgt, drf, tokens, uniforms, temperature, sigma_F, sigma_C, *, desc_out=None,
                     probs=True, workspace=None, dev_status=None, stream=None):
    """ssd_verify on sigma_{F_k,C} with the descriptors found in the same pass:
    returns dict(accept_len, bonus[, p_tok, q_tok], desc)."""
    B, K, V, drf_rows = _shapes(tgt, drf, tokens)
    dev = tgt.device
    _dev(uniforms, "uniforms", torch.float32)
    _dev(temperature, "temperature", torch.float32)
    Fs, desc_out = _sigma_args(sigma_F, K, B, desc_out, dev)
    accept_len = torch.empty(B, dtype=torch.int32, device=dev)
    bonus = torch.empty(B, dtype=torch.int32, device=dev)
    p_tok = torch.empty((B, K), dtype=torch.float32, device=dev) if probs else None
    q_tok = torch.empty((B, K), dtype=torch.float32, device=dev) if probs else None
    ws = _workspace(workspace, B, K, dev)
    _check(lib().ssd_verify_sigma(
        _ptr(tgt), _ptr(drf), _logit_dtype(tgt), B, K, V, drf_rows, _ptr(tokens), _ptr(uniforms),
        _ptr(temperature), _ptr(Fs), float(sigma_C), _ptr(desc_out), _ptr(accept_len), _ptr(bonus),
        _ptr(p_tok), _ptr(q_tok), _ptr(ws), ws.numel(),
        _ptr(_opt(dev_status, "dev_status", torch.int32)), _stream(stream)), "ssd_verify_sigma")
    out = {"accept_len": accept_len, "bonus": bonus, "desc": desc_out}
    if probs:
        out.update(p_tok=p_tok, q_tok=q_tok)
    return out


def ssd_round_sigma(tgt, drf, tokens, uniforms, temperature, sigma_F, sigma_C, F, budget, *,
                    desc_out=None, probs=True, workspace=None, dev_status=None, stream=None):
    """ssd_round on sigma_{F_k,C} with the descriptors found in the same pass: returns the
    outputs of ssd_round plus desc."""
    B, K, V, drf_rows = _shapes(tgt, drf, tokens)
    dev = tgt.device
    _dev(uniforms, "uniforms", torch.float32)
    _dev(temperature, "temperature", torch.float32)
    Fs, desc_out = _sigma_args(sigma_F, K, B, desc_out, dev)
    Fh = _F_host(F)
    o = {"accept_len": torch.empty(B, dtype=torch.int32, device=dev),
         "bonus": torch.empty(B, dtype=torch.int32, device=dev),
         "cache_tok": torch.full((B, budget), -1, dtype=torch.int32, device=dev),
         "hit": torch.empty(B, dtype=torch.uint8, device=dev),
         "slot": torch.empty(B, dtype=torch.int32, device=dev), "desc": desc_out}
    if probs:
        o["p_tok"] = torch.empty((B, K), dtype=torch.float32, device=dev)
        o["q_tok"] = torch.empty((B, K), dtype=torch.float32, device=dev)
    ws = _workspace(workspace, B, K, dev)
    _check(lib().ssd_round_sigma(
        _ptr(tgt), _ptr(drf), _logit_dtype(tgt), B, K, V, drf_rows, _ptr(tokens), _ptr(uniforms),
        _ptr(temperature), _ptr(Fs), float(sigma_C), _ptr(desc_out), _ptr(Fh), int(budget),
        _ptr(o["accept_len"]), _ptr(o["bonus"]), _ptr(o.get("p_tok")), _ptr(o.get("q_tok")),
        _ptr(o["cache_tok"]), _ptr(o["hit"]), _ptr(o["slot"]), _ptr(ws), ws.numel(),
        _ptr(_opt(dev_status, "dev_status", torch.int32)), _stream(stream)), "ssd_round_sigma")
    return o


def ssd_reshape_draft(drf, F, C, temperature_rows=None, *, want_q=False, desc=None, q_out=None,
                      dev_status=None, stream=None):
    """sigma_{F,C} descriptors of every draft row (drf [..., V] viewed as [rows, V]).

    Returns (desc [rows, 4] int32 holding {thr_val (fp32 bits), thr_id, F, C (fp32 bits)},
    q' [rows, V] fp32 or None)."""
    _dev(drf, "drf")
    V = int(drf.shape[-1])
    rows = drf.numel() // V
    dev = drf.device
    desc = desc if desc is not None else torch.empty((rows, 4), dtype=torch.int32, device=dev)
    if want_q:
        q_out = q_out if q_out is not None else torch.empty((rows, V), dtype=torch.float32, device=dev)
        _dev(temperature_rows, "temperature_rows", torch.float32)
    _check(lib().ssd_reshape_draft(
        _ptr(drf), _logit_dtype(drf), rows, V, _ptr(temperature_rows), int(F), float(C), _ptr(desc),
        _ptr(q_out if want_q else None), _ptr(_opt(dev_status, "dev_status", torch.int32)),
        _stream(stream)), "ssd_reshape_draft")
    return desc, (q_out if want_q else None)


def ssd_draft_cache(drf, tokens, F, budget, C=1.0, *, cache=True, reshape=False, cache_tok=None,
                    desc=None, dev_status=None, stream=None):
    """Draft-side cache keys and sigma_{F_k,C} descriptors from drf [B, K+1, V].

    Returns (cache_tok [B, budget] int32 or None, desc [B*K, 4] int32 or None); tokens
    [B, K] int32 (the drafted tokens left out of their segment) may be None."""
    _dev(drf, "drf")
    if drf.dim() != 3:
        raise ValueError("drf must be [B, K+1, V]")
    B, K1, V = drf.shape
    K = K1 - 1
    Fh = _F_host(F)
    if len(Fh) != K + 1:
        raise ValueError("F must have K+1 entries")
    dev = drf.device
    if tokens is not None:
        _dev(tokens, "tokens", torch.int32)
        if tuple(tokens.shape) != (B, K):
            raise ValueError("tokens must be [B, K]")
    if cache:
        cache_tok = cache_tok if cache_tok is not None else torch.empty(
            (B, budget), dtype=torch.int32, device=dev)
        _dev(cache_tok, "cache_tok", torch.int32)
        if tuple(cache_tok.shape) != (B, budget):
            raise ValueError("cache_tok must be [B, budget]")
    else:
        cache_tok = None
    if reshape:
        desc = desc if desc is not None else torch.empty((B * K, 4), dtype=torch.int32, device=dev)
        _dev(desc, "desc", torch.int32)
        if desc.numel() != B * K * 4:
            raise ValueError("desc must hold B*K descriptors")
    else:
        desc = None
    _check(lib().ssd_draft_cache(
        _ptr(drf), _logit_dtype(drf), B, K, V, _ptr(tokens), _ptr(Fh), int(budget), float(C),
        _ptr(cache_tok), _ptr(desc), _ptr(_opt(dev_status, "dev_status", torch.int32)),
        _stream(stream)), "ssd_draft_cache")
    return cache_tok, desc


def desc_fields(desc: torch.Tensor):
    """Decodes reshape descriptors: (thr_val fp32, thr_id int32, F int32, C fp32) tensors."""
    return desc[:, 0].view(torch.float32), desc[:, 1], desc[:, 2], desc[:, 3].view(torch.float32)


# ---------------------------------------------------------------------------
# The loop around a round: the paged 8-bit cache and truncated sampling.
# ---------------------------------------------------------------------------

# These calls take microseconds on the GPU, so their Python side counts: tensors are
# checked and turned into addresses in one go, and the current stream is looked up as a
# plain number.
try:
    _current_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:
    def _current_stream(device: int) -> int:
        return torch.cuda.current_stream(device).cuda_stream


try:
    _current_device = torch._C._cuda_getDevice
except AttributeError:
    _current_device = torch.cuda.current_device


def _stream_at(stream, t) -> int:
    if stream is None:
        return _current_stream(t.get_device())
    if not isinstance(stream, torch.cuda.Stream):
        return int(stream)
    if stream.device_index != _current_device():
        raise ValueError(f"stream is of cuda:{stream.device_index}, the current device is cuda:{_current_device()}")
    return stream.cuda_stream


def _device_of(t, name: str) -> int:
    """The device of a call's first tensor: the current one, on which the call launches."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return dev


def _not_here(t, name: str, dev: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")


def _at(t, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of that dtype, shape and device."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _not_here(t, name, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _cuda(t, name: str, dim: int, dev: int):
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _not_here(t, name, dev)
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {list(t.shape)}")
    return t.shape


def _status_at(dev_status, dev: int):
    return None if dev_status is None else _at(dev_status, "dev_status", torch.int32, dev_status.shape, dev)


def _on(stream, *made):
    """Tensors allocated here for a call on another stream than the current one: the
    allocator must not hand their memory on before that stream has used it."""
    if stream is not None:
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
        for t in made:
            if t is not None:
                t.record_stream(s)


def kv_state(B: int, max_blocks: int, num_pages: int, device=None) -> dict:
    """The state of a loop of B sequences over a cache of num_pages pages, nothing held:
    dict(seq_len, held, ring_state, ring, block_table), views of one int32 tensor
    (`buffer`), so that one copy saves or restores it."""
    head = 2 * B + 2
    buf = torch.zeros(head + num_pages + B * max_blocks, dtype=torch.int32, device=device or "cuda")
    buf[2 * B + 1] = num_pages
    buf[head:head + num_pages] = torch.arange(num_pages, dtype=torch.int32, device=buf.device)
    buf[head + num_pages:] = -1
    return {"seq_len": buf[:B], "held": buf[B:2 * B], "ring_state": buf[2 * B:head],
            "ring": buf[head:head + num_pages], "block_table": buf[head + num_pages:].view(B, max_blocks),
            "buffer": buf}


def ssd_kv_plan(seq_len, new_len, held, block_table, ring, ring_state, page_size: int, cap: int, *,
                accept_len=None, out=None, dev_status=None, stream=None):
    """Commits accept_len, and gives each sequence's new_len next tokens their pages and
    slots: updates seq_len, held, block_table, ring and ring_state in place and returns
    dict(cu_new [B+1], kv_len [B], slots [cap], positions [cap]), all int32."""
    i32, dev = torch.int32, _device_of(seq_len, "seq_len")
    B, = _cuda(seq_len, "seq_len", 1, dev)
    rows, max_blocks = _cuda(block_table, "block_table", 2, dev)
    num_pages, = _cuda(ring, "ring", 1, dev)
    cap, of_b = int(cap), (B,)
    if rows != B:
        raise ValueError("block_table must be [B, max_blocks]")
    if cap < 0:
        raise ValueError("cap must not be negative")
    o, made, at = ({} if out is None else dict(out)), [], []
    for name, n in (("cu_new", B + 1), ("kv_len", B), ("slots", cap), ("positions", cap)):
        t = o.get(name)
        if t is None:
            t = o[name] = torch.empty(n, dtype=i32, device=seq_len.device)
            made.append(t)
            at.append(t.data_ptr())
        else:
            at.append(_at(t, name, i32, (n,), dev))
    _check(lib().ssd_kv_plan(
        _at(seq_len, "seq_len", i32, of_b, dev),
        None if accept_len is None else _at(accept_len, "accept_len", i32, of_b, dev),
        _at(new_len, "new_len", i32, of_b, dev), _at(held, "held", i32, of_b, dev), B,
        _at(block_table, "block_table", i32, (B, max_blocks), dev), max_blocks, _at(ring, "ring", i32, (num_pages,), dev),
        _at(ring_state, "ring_state", i32, (2,), dev), num_pages, int(page_size), cap, *at, _status_at(dev_status, dev),
        _stream_at(stream, seq_len)), "ssd_kv_plan")
    if stream is not None:
        _on(stream, *made)
    return o


_KV_DTYPES = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16, torch.float16: SSD_F16}


_BYTES = (torch.float8_e4m3fn, torch.uint8)


def _kv_cache(k_cache, v_cache, k_scale, v_scale, dev):
    """(num_pages, Hkv, page_size, D) and the four addresses."""
    shape = _cuda(k_cache, "k_cache", 4, dev)
    kind = k_cache.dtype
    if kind not in _BYTES:
        raise TypeError(f"k_cache must be float8_e4m3fn or uint8, got {kind}")
    blocks = shape[:2]
    return shape, (_at(k_cache, "k_cache", kind, shape, dev), _at(v_cache, "v_cache", kind, shape, dev),
                   _at(k_scale, "k_scale", torch.float32, blocks, dev), _at(v_scale, "v_scale", torch.float32, blocks, dev))


def _int32(x, name) -> int:
    x = int(x)
    if not -1 << 31 <= x < 1 << 31:     # ctypes would drop the upper bits
        raise ValueError(f"{name} does not fit in 32 bits")
    return x


def _tokens(t, name, H, D, dev):
    """(T, heads, token stride) of a [T, H, D] tensor whose heads and channels are contiguous."""
    T, heads, width = _cuda(t, name, 3, dev)
    if t.dtype not in _KV_DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if width != D or (H is not None and heads != H):
        raise ValueError(f"{name} must be [T, {'heads' if H is None else H}, {D}]")
    ld, per_head, per_channel = t.stride()
    if per_channel != 1 or (heads > 1 and per_head != D):
        raise ValueError(f"{name}: heads and channels must be contiguous")
    if T <= 1:
        ld = heads * D
    if ld < heads * D:
        raise ValueError(f"{name}: tokens overlap")
    return T, heads, ld


def ssd_kv_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, *, dev_status=None, stream=None):
    """Stores keys and values [T, Hkv, D] (views with a longer token stride are fine) at
    `slots` of the e4m3 cache, growing the touched pages' power-of-two scales in place."""
    dev = _device_of(k, "k")
    (N, H, P, D), cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    (T, _, ks), (Tv, _, vs) = _tokens(k, "k", H, D, dev), _tokens(v, "v", H, D, dev)
    if T != Tv or v.dtype is not k.dtype:
        raise ValueError("k and v must match in shape and dtype")
    _check(lib().ssd_kv_append(
        k.data_ptr(), v.data_ptr(), _KV_DTYPES[k.dtype], ks, vs, _at(slots, "slots", torch.int32, (T,), dev), T, H, D,
        *cache, N, P, _status_at(dev_status, dev), _stream_at(stream, k)), "ssd_kv_append")


def kv_workspace(device=None) -> torch.Tensor:
    """A zero-filled workspace for ssd_kv_attend (one per stream)."""
    return torch.zeros(int(lib().ssd_kv_workspace_size()), dtype=torch.uint8, device=device or "cuda")


def ssd_kv_attend(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_new, kv_len, max_new: int,
                  sm_scale: float, *, window: int = 0, out=None, workspace=None, dev_status=None, stream=None):
    """Causal attention of q [T, Hq, D] (bf16 or fp16) over the paged e4m3 cache: returns
    out [T, Hq, D].  cu_new and kv_len as from ssd_kv_plan."""
    dev = _device_of(q, "q")
    (N, Hkv, P, D), cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    T, Hq, ld = _tokens(q, "q", None, D, dev)
    B, = _cuda(kv_len, "kv_len", 1, dev)
    rows, max_blocks = _cuda(block_table, "block_table", 2, dev)
    if rows != B:
        raise ValueError("block_table must be [B, max_blocks]")
    i32, made = torch.int32, []
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
        made.append(out)
    if workspace is None:
        workspace = kv_workspace(q.device)
        made.append(workspace)
        if stream is not None:
            # its fill runs on the current stream
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
            s.wait_stream(torch.cuda.current_stream())
    _check(lib().ssd_kv_attend(
        q.data_ptr(), _KV_DTYPES[q.dtype], ld, *cache, N, P, Hq, Hkv, D,
        _at(block_table, "block_table", i32, (B, max_blocks), dev), max_blocks, _at(cu_new, "cu_new", i32, (B + 1,), dev),
        _at(kv_len, "kv_len", i32, (B,), dev), B, T, _int32(max_new, "max_new"), float(sm_scale), _int32(window, "window"),
        _at(out, "out", q.dtype, (T, Hq, D), dev), _at(workspace, "workspace", torch.uint8, workspace.shape, dev),
        workspace.numel(), _status_at(dev_status, dev), _stream_at(stream, q)), "ssd_kv_attend")
    if stream is not None:
        _on(stream, *made)
    return out


def ssd_sample(logits, temperature, uniforms, *, top_k=None, top_p=None, min_p=None, filtered=False, tokens=None,
               prob=None, dev_status=None, stream=None):
    """One token per row of logits [rows, V] (rows may be a [..., :V] view of longer ones)
    under temperature, top-k, top-p and min-p: returns dict(tokens, prob[, filtered]).
    filtered: True, or a tensor of the logits' shape and strides, for the logits with every
    dropped token at SSD_DROPPED_LOGIT (rows too low for that are copied: SSD_DEV_LOW_LOGITS)."""
    dev = _device_of(logits, "logits")
    R, V = _cuda(logits, "logits", 2, dev)
    dt = _logit_dtype(logits)
    ld, step = logits.stride()
    if R <= 1:
        ld = V
    if step != 1 or ld < V:
        raise ValueError("logits: rows must be contiguous and must not overlap")
    f32, i32, of_r, made = torch.float32, torch.int32, (R,), []
    if tokens is None:
        tokens = torch.empty(R, dtype=i32, device=logits.device)
        made.append(tokens)
    if prob is None:
        prob = torch.empty(R, dtype=f32, device=logits.device)
        made.append(prob)
    if filtered is True:
        filtered = torch.empty((R, ld), dtype=logits.dtype, device=logits.device)[:, :V]
        made.append(filtered)
    elif filtered is False:
        filtered = None
    if filtered is not None:
        if not isinstance(filtered, torch.Tensor) or filtered.get_device() != dev:
            _not_here(filtered, "filtered", dev)
        if filtered.dtype is not logits.dtype:
            raise TypeError("filtered must be a CUDA tensor of the logits' dtype")
        if filtered.shape != logits.shape or filtered.stride(1) != 1 or (R > 1 and filtered.stride(0) != ld):
            raise ValueError("filtered must have the logits' shape and strides")
    _check(lib().ssd_sample(
        logits.data_ptr(), dt, R, V, ld, _at(temperature, "temperature", f32, of_r, dev),
        None if top_k is None else _at(top_k, "top_k", i32, of_r, dev), None if top_p is None else _at(top_p, "top_p", f32, of_r, dev),
        None if min_p is None else _at(min_p, "min_p", f32, of_r, dev), _at(uniforms, "uniforms", f32, of_r, dev),
        _at(tokens, "tokens", i32, of_r, dev), _at(prob, "prob", f32, of_r, dev), None if filtered is None else filtered.data_ptr(),
        _status_at(dev_status, dev), _stream_at(stream, logits)), "ssd_sample")
    if stream is not None:
        _on(stream, *made)
    out = {"tokens": tokens, "prob": prob}
    if filtered is not None:
        out["filtered"] = filtered
    return out


# ---------------------------------------------------------------------------
# A tree of drafted tokens.
# ---------------------------------------------------------------------------

def rope_turns(inv_freq, device=None) -> torch.Tensor:
    """Rotary frequencies (radians for each position, a tensor or a list) in the form that
    ssd_qk_rope takes: int64 fractions of a turn in units of 2^-64.  Made once for a model."""
    if isinstance(inv_freq, torch.Tensor):
        device = device or inv_freq.device
        inv_freq = inv_freq.detach().to(device="cpu", dtype=torch.float64).flatten().tolist()
    full = 1 << 64
    out = []
    for f in inv_freq:
        v = int(round(math.fmod(float(f) / (2 * math.pi), 1.0) * full)) % full
        out.append(v - full if v >= full // 2 else v)
    return torch.tensor(out, dtype=torch.int64, device=device or "cuda")


def ssd_qk_rope(q, k, positions, turns, *, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                q_out=None, k_out=None, stream=None):
    """Norms each head of q [T, Hq, D] and k [T, Hkv, D] (with q_weight and k_weight [D] fp32) and turns its
    first 2 * len(turns) channels by positions [T]: returns (q_out, k_out).  All four may be views with a
    longer token stride; q_out=q, k_out=k works in place."""
    dev = _device_of(q, "q")
    D = q.shape[-1] if q.dim() == 3 else 0
    (T, Hq, qs), (Tk, Hkv, ks) = _tokens(q, "q", None, D, dev), _tokens(k, "k", None, D, dev)
    if T != Tk or k.dtype is not q.dtype:
        raise ValueError("q and k must match in tokens and dtype")
    made = []
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
        made.append(q_out)
        qos = Hq * D
    else:
        To, _, qos = _tokens(q_out, "q_out", Hq, D, dev)
        if To != T or q_out.dtype is not q.dtype:
            raise ValueError("q_out must match q in tokens and dtype")
    if k_out is None:
        k_out = torch.empty((T, Hkv, D), dtype=q.dtype, device=q.device)
        made.append(k_out)
        kos = Hkv * D
    else:
        To, _, kos = _tokens(k_out, "k_out", Hkv, D, dev)
        if To != T or k_out.dtype is not q.dtype:
            raise ValueError("k_out must match k in tokens and dtype")
    R, = _cuda(turns, "turns", 1, dev)
    f32 = torch.float32
    _check(lib().ssd_qk_rope(
        q.data_ptr(), k.data_ptr(), _KV_DTYPES[q.dtype], qs, ks, T, Hq, Hkv, D,
        None if q_weight is None else _at(q_weight, "q_weight", f32, (D,), dev),
        None if k_weight is None else _at(k_weight, "k_weight", f32, (D,), dev), float(eps),
        _at(positions, "positions", torch.int32, (T,), dev), _at(turns, "turns", torch.int64, (R,), dev), 2 * R,
        1 if interleaved else 0, q_out.data_ptr(), k_out.data_ptr(), qos, kos, _stream_at(stream, q)), "ssd_qk_rope")
    if stream is not None:
        _on(stream, *made)
    return q_out, k_out


def ssd_tree_plan(parent, cu_new, seq_len, max_new: int, *, out=None, dev_status=None, stream=None):
    """Masks and positions of the trees that parent [T] describes (index of each node's parent among its
    sequence's nodes, -1 for a root): returns dict(positions [T], mask [T, ceil(max_new / 32)]), int32."""
    i32, dev = torch.int32, _device_of(parent, "parent")
    T, = _cuda(parent, "parent", 1, dev)
    B, = _cuda(seq_len, "seq_len", 1, dev)
    max_new = int(max_new)
    W = (max_new + 31) // 32
    if W < 1:
        raise ValueError("max_new must be positive")
    _check(SSD_OK if max_new <= SSD_TREE_MAX else SSD_ERR_UNSUPPORTED, "ssd_tree_plan")      # (before a mask of that size is made)
    o, made = ({} if out is None else dict(out)), []
    for name, shape in (("positions", (T,)), ("mask", (T, W))):
        if o.get(name) is None:
            o[name] = torch.empty(shape, dtype=i32, device=parent.device)
            made.append(o[name])
    _check(lib().ssd_tree_plan(
        _at(parent, "parent", i32, (T,), dev), _at(cu_new, "cu_new", i32, (B + 1,), dev), _at(seq_len, "seq_len", i32, (B,), dev), B, T,
        max_new, _at(o["positions"], "positions", i32, (T,), dev), _at(o["mask"], "mask", i32, (T, W), dev),
        _status_at(dev_status, dev), _stream_at(stream, parent)), "ssd_tree_plan")
    if stream is not None:
        _on(stream, *made)
    return o


def kv_tree_workspace(device=None) -> torch.Tensor:
    """A zero-filled workspace for ssd_kv_attend_tree (one per stream)."""
    return torch.zeros(int(lib().ssd_kv_tree_workspace_size()), dtype=torch.uint8, device=device or "cuda")


def ssd_kv_attend_tree(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_new, kv_len, mask, max_new: int, sm_scale: float, *,
                       window: int = 0, out=None, workspace=None, dev_status=None, stream=None):
    """Attention of trees of new tokens, q [T, Hq, D] (bf16 or fp16), over the paged e4m3 cache: each sees the
    positions before its tree and the nodes of its row of mask [T, ceil(max_new / 32)] (ssd_tree_plan).
    Returns out [T, Hq, D]."""
    dev = _device_of(q, "q")
    (N, Hkv, P, D), cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    T, Hq, ld = _tokens(q, "q", None, D, dev)
    B, = _cuda(kv_len, "kv_len", 1, dev)
    rows, max_blocks = _cuda(block_table, "block_table", 2, dev)
    if rows != B:
        raise ValueError("block_table must be [B, max_blocks]")
    i32, made = torch.int32, []
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
        made.append(out)
    if workspace is None:
        workspace = kv_tree_workspace(q.device)
        made.append(workspace)
        if stream is not None:
            # its fill runs on the current stream
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
            s.wait_stream(torch.cuda.current_stream())
    _check(lib().ssd_kv_attend_tree(
        q.data_ptr(), _KV_DTYPES[q.dtype], ld, *cache, N, P, Hq, Hkv, D,
        _at(block_table, "block_table", i32, (B, max_blocks), dev), max_blocks, _at(cu_new, "cu_new", i32, (B + 1,), dev),
        _at(kv_len, "kv_len", i32, (B,), dev), _at(mask, "mask", i32, (T, (int(max_new) + 31) // 32), dev), B, T,
        _int32(max_new, "max_new"), float(sm_scale), _int32(window, "window"), _at(out, "out", q.dtype, (T, Hq, D), dev),
        _at(workspace, "workspace", torch.uint8, workspace.shape, dev), workspace.numel(), _status_at(dev_status, dev),
        _stream_at(stream, q)), "ssd_kv_attend_tree")
    if stream is not None:
        _on(stream, *made)
    return out


def ssd_tree_accept(parent, tokens, sampled, cu_new, max_new: int, max_path: int, *, out=None, dev_status=None, stream=None):
    """Follows the draws `sampled` [T] at the nodes of trees (parent, tokens [T]) from each node 0 down: returns
    dict(accept_len [B], bonus [B], path [B, max_path]), int32."""
    i32, dev = torch.int32, _device_of(parent, "parent")
    T, = _cuda(parent, "parent", 1, dev)
    B = _cuda(cu_new, "cu_new", 1, dev)[0] - 1
    J, of_t, of_b = int(max_path), (T,), (B,)
    if B < 0 or J < 0:
        raise ValueError("cu_new must be [B+1] and max_path positive")
    _check(SSD_OK if J <= SSD_MAX_K + 1 else SSD_ERR_INVALID_ARG, "ssd_tree_accept")         # (before a path of that size is made)
    o, made = ({} if out is None else dict(out)), []
    for name, shape in (("accept_len", of_b), ("bonus", of_b), ("path", (B, J))):
        if o.get(name) is None:
            o[name] = torch.empty(shape, dtype=i32, device=parent.device)
            made.append(o[name])
    _check(lib().ssd_tree_accept(
        _at(parent, "parent", i32, of_t, dev), _at(tokens, "tokens", i32, of_t, dev), _at(sampled, "sampled", i32, of_t, dev),
        _at(cu_new, "cu_new", i32, (B + 1,), dev), B, T, _int32(max_new, "max_new"), J, _at(o["accept_len"], "accept_len", i32, of_b, dev),
        _at(o["bonus"], "bonus", i32, of_b, dev), _at(o["path"], "path", i32, (B, J), dev), _status_at(dev_status, dev),
        _stream_at(stream, parent)), "ssd_tree_accept")
    if stream is not None:
        _on(stream, *made)
    return o


def ssd_kv_compact(path, accept_len, seq_len, block_table, k_cache, v_cache, k_scale, v_scale, *, dev_status=None, stream=None):
    """Moves the keys and values of the accepted paths [B, max_path] to the rows from seq_len [B] on, in place;
    pages that tokens of others come into grow their scales as in ssd_kv_append."""
    i32, dev = torch.int32, _device_of(path, "path")
    B, J = _cuda(path, "path", 2, dev)
    (N, H, P, D), cache = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    max_blocks = _cuda(block_table, "block_table", 2, dev)[1]
    _check(lib().ssd_kv_compact(
        _at(path, "path", i32, (B, J), dev), _at(accept_len, "accept_len", i32, (B,), dev), _at(seq_len, "seq_len", i32, (B,), dev), B, J,
        _at(block_table, "block_table", i32, (B, max_blocks), dev), max_blocks, H, D, *cache, N, P, _status_at(dev_status, dev),
        _stream_at(stream, path)), "ssd_kv_compact")
