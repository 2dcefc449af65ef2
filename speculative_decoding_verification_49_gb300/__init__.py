"""GB300 speculative-sampling verify step.

Python binding of ``libspecverify.so`` (the CUDA kernels behind the C ABI in
``include/spec_verify.h``, and for the KV cache ``include/spec_verify_cache.h``).
The functions named ``spec_verify_*`` mirror the
C entry points one to one and take raw device pointers; ``SpecVerify`` is a
convenience wrapper that takes torch tensors and only marshals arguments.
Every step of the verify computation runs in the CUDA library: there is no
Python or CPU fallback, and importing a missing library raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

from .build import LIBRARY

SV_OK = 0
SV_ERR_INVALID_ARG = 1
SV_ERR_SHAPE = 2
SV_ERR_DTYPE = 3
SV_ERR_CUDA = 4
SV_ERR_OOM = 5
SV_ERR_BAD_TOKEN = 6
SV_ERR_BAD_VALUE = 7
SV_ERR_TIMEOUT = 8
SV_ERR_TOO_LARGE = 9
SV_ERR_BAD_TREE = 10

SV_F32 = 0
SV_BF16 = 1

_P = ctypes.c_void_p
_I = ctypes.c_int

# (name, restype, argtypes) of every exported entry point
_SIGNATURES = [
    ("spec_verify_create", _I, [ctypes.POINTER(_P), _I, _I, _I, _I, _I]),
    ("spec_verify_run", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P]),
    ("spec_verify_run_debug", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    ("spec_verify_get_status", _I, [_P]),
    ("spec_verify_set_cluster_size", _I, [_P, _I]),
    ("spec_verify_cluster_size", _I, [_P, _I, _I]),
    ("spec_verify_set_fused_logits", _I, [_P, _I]),
    ("spec_verify_error_string", ctypes.c_char_p, [_I]),
    ("spec_verify_destroy", None, [_P]),
    ("spec_verify_run_noalloc", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    ("spec_verify_profile", _I, [_P, _I]),
    ("spec_verify_acceptance_counts", _I, [_P, ctypes.POINTER(ctypes.c_uint64), _I, _I]),
    ("spec_verify_profile_read", _I, [_P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                                      ctypes.POINTER(_I)]),
    ("spec_verify_kv_commit", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_size_t, _P]),
    ("spec_verify_tree_run", _I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
    ("spec_verify_lm_head_logits", _I, [_P, _P, _I, _I, _I, _P, _P]),
    ("spec_verify_selftest_timeout", _I, [_I, ctypes.POINTER(_I), _P]),
    ("spec_verify_run_fused", _I, [_P, _P, _P, _I, _P, _P, _I, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
]

SV_KV_OVERFLOW = 1
SV_KV_BAD_COUNT = 2

# the entry points of include/spec_verify_cache.h
_CACHE_SIGNATURES = [
    ("spec_verify_kv_commit_path", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    ("spec_verify_kv_read", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    ("spec_verify_attention_workspace", _I, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_int64)]),
    ("spec_verify_attention", _I, [ctypes.c_char_p, _P]),
]

SV_KV_BAD_PATH = 4
SV_KV_NONFINITE = 8

SV_KV_BF16 = 0
SV_KV_E4M3 = 1

SV_ATTN_BAD_LEN = 1
SV_ATTN_BAD_TREE = 2
SV_ATTN_TIMEOUT = 4

_lib = None


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__(f"{where}: {spec_verify_error_string(status)}" if where else spec_verify_error_string(status))


def load() -> ctypes.CDLL:
    """Load the CUDA library; raises ImportError when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY):
            raise ImportError(f"{LIBRARY} is missing: build it with "
                              "`python -m speculative_decoding_verification_49_gb300.build`")
        lib = ctypes.CDLL(LIBRARY)
        for name, res, args in _SIGNATURES + _CACHE_SIGNATURES:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def exported_names():
    """The entry points of include/spec_verify.h."""
    return [s[0] for s in _SIGNATURES]


def exported_cache_names():
    """The entry points of include/spec_verify_cache.h."""
    return [s[0] for s in _CACHE_SIGNATURES]


# ---- one-to-one wrappers of the C ABI (raw pointers as Python ints) ---------

def spec_verify_create(device: int, max_B: int, max_N: int, V: int, dtype: int) -> int:
    ctx = _P()
    st = load().spec_verify_create(ctypes.byref(ctx), device, max_B, max_N, V, dtype)
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_create")
    return ctx.value


def spec_verify_run(ctx, target, draft, draft_tokens, uniforms, temperature, greedy, B, N,
                    out_tokens, num_accepted, stream) -> int:
    return load().spec_verify_run(ctx, target, draft, draft_tokens, uniforms, temperature,
                                  int(greedy), B, N, out_tokens, num_accepted, stream)


def spec_verify_run_debug(ctx, target, draft, draft_tokens, uniforms, temperature, greedy, B, N,
                          out_tokens, num_accepted, stream, q_at_draft, p_at_draft,
                          target_row_stats, draft_row_stats, ratio_at_draft=None) -> int:
    return load().spec_verify_run_debug(ctx, target, draft, draft_tokens, uniforms, temperature,
                                        int(greedy), B, N, out_tokens, num_accepted, stream,
                                        q_at_draft, p_at_draft, target_row_stats, draft_row_stats,
                                        ratio_at_draft)


def spec_verify_get_status(ctx) -> int:
    return load().spec_verify_get_status(ctx)


def spec_verify_set_cluster_size(ctx, cluster_size: int) -> int:
    return load().spec_verify_set_cluster_size(ctx, cluster_size)


def spec_verify_cluster_size(ctx, B: int, N: int) -> int:
    return load().spec_verify_cluster_size(ctx, B, N)


def spec_verify_set_fused_logits(ctx, keep: bool) -> int:
    return load().spec_verify_set_fused_logits(ctx, int(bool(keep)))


def spec_verify_error_string(status: int) -> str:
    return load().spec_verify_error_string(status).decode()


def spec_verify_destroy(ctx) -> None:
    load().spec_verify_destroy(ctx)


def spec_verify_run_noalloc(target, draft, draft_tokens, uniforms, temperature, greedy, B, N, V, dtype,
                            out_tokens, num_accepted, stream) -> int:
    """Context-free variant that allocates nothing: scratch is a fixed array
    inside the library (B <= 2048, B*(N+1) <= 16384,
    B*ceil(V*elt/4KiB) <= 32768), shared by every call on
    the device, so calls must not overlap on the GPU."""
    return load().spec_verify_run_noalloc(target, draft, draft_tokens, uniforms, temperature,
                                          int(greedy), B, N, V, dtype, out_tokens, num_accepted, stream)


def spec_verify_acceptance_counts(ctx, ncounts: int, reset: bool = False):
    """(status, counts): counts[k] sequences that accepted k drafts, the last
    entry invalid sequences."""
    arr = (ctypes.c_uint64 * ncounts)()
    st = load().spec_verify_acceptance_counts(ctx, arr, ncounts, int(bool(reset)))
    return st, list(arr)


def spec_verify_profile(ctx, enable: bool) -> int:
    return load().spec_verify_profile(ctx, int(bool(enable)))


def spec_verify_profile_read(ctx):
    """(status, ms_rows, ms_sample, runs) summed over the profiled runs."""
    a, b, n = ctypes.c_double(), ctypes.c_double(), _I()
    st = load().spec_verify_profile_read(ctx, ctypes.byref(a), ctypes.byref(b), ctypes.byref(n))
    return st, a.value, b.value, n.value


def spec_verify_tree_run(ctx, target, draft, parent, draft_tokens, uniforms, temperature, greedy, B, M,
                         out_tokens, path_nodes, num_accepted, target_row_stats, draft_row_stats, ratio_at_node,
                         stream) -> int:
    """Verify B candidate trees of M+1 nodes (device pointers; asynchronous)."""
    return load().spec_verify_tree_run(ctx, target, draft, parent, draft_tokens, uniforms, temperature,
                                       int(greedy), B, M, out_tokens, path_nodes, num_accepted,
                                       target_row_stats, draft_row_stats, ratio_at_node, stream)


def spec_verify_kv_commit(scratch, cache, cache_len, num_accepted, status, planes, B, N, max_len, row_bytes,
                          stream) -> int:
    """Append each sequence's first num_accepted scratch KV rows to its cache
    and advance cache_len (device pointers; asynchronous on stream)."""
    return load().spec_verify_kv_commit(scratch, cache, cache_len, num_accepted, status, planes, B, N,
                                        max_len, row_bytes, stream)


def spec_verify_kv_commit_path(rows, cache, scale, cache_len, out_len, num_accepted, path, status, planes, B, T,
                               lead, max_len, heads, head_dim, format, stream) -> int:
    """Append each sequence's lead and accepted rows to its cache, in bf16 or
    quantised to e4m3, and write the new lengths (device pointers; asynchronous)."""
    return load().spec_verify_kv_commit_path(rows, cache, scale, cache_len, out_len, num_accepted, path, status,
                                             planes, B, T, lead, max_len, heads, head_dim, format, stream)


def spec_verify_kv_read(cache, scale, cache_len, start, out, status, planes, B, n, max_len, heads, head_dim,
                        stream) -> int:
    """Read rows of an e4m3 cache back as bf16 (device pointers; asynchronous)."""
    return load().spec_verify_kv_read(cache, scale, cache_len, start, out, status, planes, B, n, max_len, heads,
                                      head_dim, stream)


# sv_attention_args: 17 pointers, the workspace's size, 4 strides, 8 sizes, the softmax scale
_ATTENTION_ARGS = struct.Struct("=17Q1q4q8qd")


def spec_verify_attention_workspace(args: bytes):
    """(status, bytes) for packed sv_attention_args."""
    n = ctypes.c_int64(0)
    st = load().spec_verify_attention_workspace(args, ctypes.byref(n))
    return st, n.value


def spec_verify_attention(args: bytes, stream) -> int:
    """The verifier's attention, from packed sv_attention_args (asynchronous)."""
    return load().spec_verify_attention(args, stream)


# ---- torch convenience wrapper -------------------------------------------------

def _ptr(t):
    return None if t is None else t.data_ptr()


class SpecVerify:
    """A context plus argument checks for torch tensors on one CUDA device.

    ``run`` enqueues the verify step on the current torch stream (or the
    given one) and returns (out_tokens [B, N+1] int32, num_accepted [B] int32)
    without synchronising.
    """

    def __init__(self, max_B: int, max_N: int, V: int, dtype: str = "bf16", device: int = 0):
        self.max_B, self.max_N, self.V, self.device = max_B, max_N, V, device
        self.dtype = dtype
        self.ctx = spec_verify_create(device, max_B, max_N, V, SV_BF16 if dtype == "bf16" else SV_F32)

    def close(self):
        if getattr(self, "ctx", None):
            spec_verify_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_cluster_size(self, c: int):
        st = spec_verify_set_cluster_size(self.ctx, c)
        if st != SV_OK:
            raise SpecVerifyError(st, "spec_verify_set_cluster_size")

    def cluster_size(self, B: int, N: int) -> int:
        return spec_verify_cluster_size(self.ctx, B, N)

    def set_fused_logits(self, keep: bool):
        """run_fused: write every verifier row's float32 logits from the
        statistics epilogue and read back the sampled rows (keep=True, the
        default), or keep them out of HBM and recompute the sampled verifier
        rows; the sampled draft rows are recomputed either way."""
        st = spec_verify_set_fused_logits(self.ctx, keep)
        if st != SV_OK:
            raise SpecVerifyError(st, "spec_verify_set_fused_logits")

    def status(self) -> int:
        return spec_verify_get_status(self.ctx)

    def acceptance_counts(self, reset: bool = False):
        """counts[k] = sequences that accepted k drafts (k = 0..max_N) since the
        last reset; counts[max_N + 1] = invalid sequences."""
        st, counts = spec_verify_acceptance_counts(self.ctx, self.max_N + 2, reset)
        if st != SV_OK:
            raise SpecVerifyError(st, "spec_verify_acceptance_counts")
        return counts

    def profile(self, enable: bool):
        st = spec_verify_profile(self.ctx, enable)
        if st != SV_OK:
            raise SpecVerifyError(st, "spec_verify_profile")

    def profile_read(self):
        """(ms in the row kernel, ms in the sampling kernel, runs)."""
        st, a, b, n = spec_verify_profile_read(self.ctx)
        if st != SV_OK:
            raise SpecVerifyError(st, "spec_verify_profile_read")
        return a, b, n

    def _check(self, target, draft, draft_tokens, uniforms, temperature, greedy):
        import torch
        want = torch.bfloat16 if self.dtype == "bf16" else torch.float32
        B, N1, V = target.shape
        N = N1 - 1
        assert V == self.V and target.dtype == want and target.is_contiguous() and target.is_cuda
        if draft is not None:
            assert draft.shape == (B, N, V) and draft.dtype == want and draft.is_contiguous()
        if draft_tokens is not None:
            assert draft_tokens.shape == (B, N) and draft_tokens.dtype == torch.int32
            assert draft_tokens.is_contiguous()
        if uniforms is not None:
            assert uniforms.shape == (B, N + 1) and uniforms.dtype == torch.float32
            assert uniforms.is_contiguous()
        if temperature is not None:
            assert temperature.shape == (B,) and temperature.dtype == torch.float32
        return B, N

    def run(self, target, draft, draft_tokens, uniforms, temperature, greedy=False,
            out_tokens=None, num_accepted=None, stream=None, debug=None):
        import torch
        B, N = self._check(target, draft, draft_tokens, uniforms, temperature, greedy)
        dev = target.device
        if out_tokens is None:
            out_tokens = torch.empty((B, N + 1), dtype=torch.int32, device=dev)
        if num_accepted is None:
            num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        args = (self.ctx, _ptr(target), _ptr(draft), _ptr(draft_tokens), _ptr(uniforms),
                _ptr(temperature), int(bool(greedy)), B, N, _ptr(out_tokens), _ptr(num_accepted),
                s.cuda_stream)
        if debug is None:
            st = spec_verify_run(*args)
        else:
            st = spec_verify_run_debug(*args, _ptr(debug.get("q_at_draft")), _ptr(debug.get("p_at_draft")),
                                       _ptr(debug.get("target_row_stats")),
                                       _ptr(debug.get("draft_row_stats")), _ptr(debug.get("ratio_at_draft")))
        if st != SV_OK:
            raise SpecVerifyError(st, "spec_verify_run")
        return out_tokens, num_accepted

    def tree_run(self, target, draft, parent, tokens, uniforms, temperature, greedy=False, out_tokens=None,
                 path_nodes=None, num_accepted=None, stream=None, stats=None):
        """Tree verification; returns (out_tokens [B, M+1], path_nodes [B, M+1],
        num_accepted [B]) without synchronising.  ``stats`` may hold
        "target_row_stats" / "draft_row_stats" float32 [B, M+1, 2] tensors and
        "ratio_at_node" float32 [B, M+1] (the ratio each tested child's
        uniform was compared with)."""
        import torch
        B, M1, V = target.shape
        M = M1 - 1
        want = torch.bfloat16 if self.dtype == "bf16" else torch.float32
        if target.dtype != want or V != self.V or not target.is_contiguous():
            raise ValueError("target logits must be contiguous [B, M+1, V] of the context's dtype")
        if draft is not None and (draft.shape != target.shape or draft.dtype != want or not draft.is_contiguous()):
            raise ValueError("draft logits must match the target's shape and dtype")
        for name, t, dt in (("parent", parent, torch.int32), ("tokens", tokens, torch.int32),
                            ("uniforms", uniforms, torch.float32)):
            if t is not None and (t.shape != (B, M + 1) or t.dtype != dt or not t.is_contiguous()):
                raise ValueError(f"{name} must be contiguous {dt} of shape ({B}, {M + 1})")
        dev = target.device
        if out_tokens is None:
            out_tokens = torch.empty((B, M + 1), dtype=torch.int32, device=dev)
        if path_nodes is None:
            path_nodes = torch.empty((B, M + 1), dtype=torch.int32, device=dev)
        if num_accepted is None:
            num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        stats = stats or {}
        st = spec_verify_tree_run(self.ctx, _ptr(target), _ptr(draft), _ptr(parent), _ptr(tokens), _ptr(uniforms),
                                  _ptr(temperature), greedy, B, M, _ptr(out_tokens), _ptr(path_nodes),
                                  _ptr(num_accepted), _ptr(stats.get("target_row_stats")),
                                  _ptr(stats.get("draft_row_stats")), _ptr(stats.get("ratio_at_node")),
                                  s.cuda_stream)
        if st != SV_OK:
            raise SpecVerifyError(st, "spec_verify_tree_run")
        return out_tokens, path_nodes, num_accepted

    def run_fused(self, target_hidden, target_weight, draft_hidden, draft_weight, draft_tokens, uniforms,
                  temperature, greedy=False, out_tokens=None, num_accepted=None, stream=None, stats=None):
        """The verify step fused into the LM-head products (context dtype
        "f32"): hidden states [rows, K] and weights [V, K] in bf16; returns
        (out_tokens, num_accepted) without synchronising."""
        import torch
        Kt = target_hidden.shape[1]
        N = draft_tokens.shape[1]
        B = target_hidden.shape[0] // (N + 1)
        Kd = draft_hidden.shape[1] if draft_hidden is not None else 0
        for t in (target_hidden, target_weight, draft_hidden, draft_weight):
            if t is not None and (t.dtype != torch.bfloat16 or not t.is_contiguous()):
                raise ValueError("hidden states and weights must be contiguous bf16")
        dev = target_hidden.device
        if out_tokens is None:
            out_tokens = torch.empty((B, N + 1), dtype=torch.int32, device=dev)
        if num_accepted is None:
            num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        stats = stats or {}
        st = load().spec_verify_run_fused(
            self.ctx, _ptr(target_hidden), _ptr(target_weight), Kt, _ptr(draft_hidden), _ptr(draft_weight), Kd,
            _ptr(draft_tokens), _ptr(uniforms), _ptr(temperature), int(bool(greedy)), B, N, _ptr(out_tokens),
            _ptr(num_accepted), _ptr(stats.get("target_row_stats")), _ptr(stats.get("draft_row_stats")),
            _ptr(stats.get("ratio_at_draft")), s.cuda_stream)
        if st != SV_OK:
            raise SpecVerifyError(st, "spec_verify_run_fused")
        return out_tokens, num_accepted

    def debug_buffers(self, B: int, N: int, device="cuda"):
        import torch
        return {
            "q_at_draft": torch.full((B, N), float("nan"), device=device),
            "p_at_draft": torch.full((B, N), float("nan"), device=device),
            "target_row_stats": torch.full((B, N + 1, 2), float("nan"), device=device),
            "draft_row_stats": torch.full((B, N, 2), float("nan"), device=device),
            "ratio_at_draft": torch.full((B, N), float("nan"), device=device),
        }


def kv_commit(scratch, cache, cache_len, num_accepted, status=None, stream=None):
    """Torch front end of spec_verify_kv_commit.

    scratch [P, B, N, *row] and cache [P, B, max_len, *row] are contiguous
    CUDA tensors of one dtype (a row is one token's entry in one plane, e.g.
    [kv_heads, head_dim]); cache_len and num_accepted are int32 [B]; status is
    an optional int32 [1] that collects SV_KV_* bits.  Enqueues on the
    current torch stream (or ``stream``) and does not synchronise."""
    import torch
    if scratch.dtype != cache.dtype or scratch.shape[:2] != cache.shape[:2] or scratch.shape[3:] != cache.shape[3:]:
        raise ValueError(f"scratch {tuple(scratch.shape)} and cache {tuple(cache.shape)} do not match")
    for name, t in (("scratch", scratch), ("cache", cache)):
        if not t.is_cuda or not t.is_contiguous() or t.dim() < 3:
            raise ValueError(f"{name} must be a contiguous CUDA tensor [P, B, rows, ...]")
    P, B, N = scratch.shape[:3]
    max_len = cache.shape[2]
    for name, t in (("cache_len", cache_len), ("num_accepted", num_accepted)):
        if t.dtype != torch.int32 or t.shape != (B,) or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of shape ({B},)")
    row_bytes = math.prod(cache.shape[3:]) * cache.element_size()
    s = stream if stream is not None else torch.cuda.current_stream(cache.device)
    st = spec_verify_kv_commit(_ptr(scratch) if N else None, _ptr(cache), _ptr(cache_len), _ptr(num_accepted),
                               _ptr(status), P, B, N, max_len, row_bytes, s.cuda_stream)
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_kv_commit")


def _kv_format(cache, scale, what):
    """The sv_kv_format of a cache tensor, its scale tensor checked: uint8, one byte a (row, head)."""
    import torch
    if cache.dtype is torch.bfloat16:
        if scale is not None:
            raise ValueError(f"a bf16 {what} has no scales")
        return SV_KV_BF16
    if cache.dtype is not torch.float8_e4m3fn:
        raise ValueError(f"{what} must be bfloat16 or float8_e4m3fn, got {cache.dtype}")
    if scale is None or scale.dtype is not torch.uint8 or scale.shape != cache.shape[:-1] \
            or not scale.is_contiguous() or scale.get_device() != cache.get_device():
        raise ValueError(f"an e4m3 {what} needs contiguous uint8 scales of shape {tuple(cache.shape[:-1])}")
    return SV_KV_E4M3


def _int32(name, t, shape, index):
    """t is contiguous int32 of that shape on CUDA device ``index``."""
    import torch
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on cuda:{index}")


def _on(index, call, *args):
    """call(*args) with CUDA device ``index`` current."""
    import torch
    if torch.cuda.current_device() == index:
        return call(*args)
    with torch.cuda.device(index):
        return call(*args)


def _raw_stream(index, stream):
    """The cudaStream_t of ``stream``, or of the device's current one."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def kv_commit_path(rows, cache, cache_len, num_accepted, path=None, lead=0, scale=None, out_len=None, status=None,
                   stream=None):
    """Torch front end of spec_verify_kv_commit_path: append the accepted path
    of every sequence to its cache, quantised when the cache is e4m3.

    rows [P, B, T, heads, head_dim] bf16 holds the entries of the pass's T
    tokens, cache [P, B, max_len, heads, head_dim] is bf16, or float8_e4m3fn
    with ``scale`` uint8 [P, B, max_len, heads]; cache_len and num_accepted are
    int32 [B]; ``path`` is None (a chain) or int32 [B, T], tree_run's path_nodes;
    ``lead`` rows are committed ahead of the accepted ones (1 for the pass's
    root).  The new lengths go to ``out_len``, which is returned (None:
    cache_len itself, advanced in place); ``status`` is an optional int32 [1]
    that collects SV_KV_* bits.  Enqueues on the current torch stream (or
    ``stream``) and does not synchronise."""
    import torch
    if rows.dim() != 5 or cache.dim() != 5:
        raise ValueError(f"rows {tuple(rows.shape)} and cache {tuple(cache.shape)} must have five dimensions")
    P, B, T, H, D = rows.shape
    L = cache.shape[2]
    dev = cache.get_device()
    if cache.shape != (P, B, L, H, D):
        raise ValueError(f"rows {tuple(rows.shape)} and cache {tuple(cache.shape)} do not match")
    if rows.dtype is not torch.bfloat16 or not rows.is_contiguous() or not cache.is_contiguous() or dev < 0 \
            or rows.get_device() != dev:
        raise ValueError("rows must be bfloat16, rows and cache contiguous on one CUDA device")
    fmt = _kv_format(cache, scale, "cache")
    if out_len is None:
        out_len = cache_len
    else:
        _int32("out_len", out_len, (B,), dev)
    _int32("cache_len", cache_len, (B,), dev)
    _int32("num_accepted", num_accepted, (B,), dev)
    if path is not None:
        _int32("path", path, (B, T), dev)
    if status is not None:
        _int32("status", status, (1,), dev)
    st = _on(dev, spec_verify_kv_commit_path, rows.data_ptr(), cache.data_ptr(), _ptr(scale), cache_len.data_ptr(),
             out_len.data_ptr(), num_accepted.data_ptr(), _ptr(path), _ptr(status), P, B, T, lead, L, H, D, fmt,
             _raw_stream(dev, stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_kv_commit_path")
    return out_len


def kv_read(cache, scale, cache_len, start=None, rows=None, out=None, status=None, stream=None):
    """Torch front end of spec_verify_kv_read: the rows start[b] (0 without
    ``start``) .. cache_len[b] - 1 of an e4m3 cache [P, B, max_len, heads,
    head_dim] as bf16, at most ``rows`` of them (max_len without it), in
    ``out`` [P, B, rows, heads, head_dim] (zeros where a new one is made; rows
    past a sequence's last one are left as they were).  Enqueues on the
    current torch stream (or ``stream``) and does not synchronise."""
    import torch
    dev = cache.get_device()
    if cache.dim() != 5 or not cache.is_contiguous() or dev < 0 or cache.dtype is not torch.float8_e4m3fn:
        raise ValueError("cache must be a contiguous float8_e4m3fn CUDA tensor [P, B, max_len, heads, head_dim]")
    _kv_format(cache, scale, "cache")
    P, B, L, H, D = cache.shape
    if out is None:
        with torch.cuda.stream(stream):
            out = torch.zeros((P, B, L if rows is None else rows, H, D), dtype=torch.bfloat16, device=cache.device)
    n = out.shape[2] if out.dim() == 5 else -1
    if out.shape != (P, B, n, H, D) or (rows is not None and n != rows) or out.dtype is not torch.bfloat16 \
            or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out must be contiguous bfloat16 [P, B, rows, heads, head_dim] on the cache's device")
    _int32("cache_len", cache_len, (B,), dev)
    if start is not None:
        _int32("start", start, (B,), dev)
    if status is not None:
        _int32("status", status, (1,), dev)
    st = _on(dev, spec_verify_kv_read, cache.data_ptr(), scale.data_ptr(), cache_len.data_ptr(), _ptr(start),
             out.data_ptr(), _ptr(status), P, B, n, L, H, D, _raw_stream(dev, stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_kv_read")
    return out


def _tokens(name, t, shape, index):
    """Strides (between sequences, between tokens) of a bf16 [B, T, heads, head_dim] tensor whose last two
    dimensions are contiguous."""
    import torch
    if t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name} must be bfloat16 {tuple(shape)} on cuda:{index}, got {t.dtype} {tuple(t.shape)}")
    sb, st, sh, sd = t.stride()
    if (sd != 1 and shape[3] > 1) or (sh != shape[3] and shape[2] > 1):
        raise ValueError(f"{name}'s heads and head_dim must be contiguous")
    return sb if shape[0] > 1 else 0, st if shape[1] > 1 else 0


@functools.lru_cache(maxsize=1024)
def _attention_bytes(B, T, Hq, H, D, L, Lp, fmt):
    """Workspace of an attention call: arithmetic on its sizes."""
    st, n = spec_verify_attention_workspace(_ATTENTION_ARGS.pack(*(0,) * 22, B, T, Hq, H, D, L, Lp, fmt, 1.0))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_attention")
    return n


def verify_attention(q, k_cache, v_cache, cache_len, k_new=None, v_new=None, parent=None, k_prefix=None,
                     v_prefix=None, k_scale=None, v_scale=None, k_prefix_scale=None, v_prefix_scale=None, scale=None,
                     out=None, lse=None, status=None, stream=None):
    """Torch front end of spec_verify_attention: the attention of the T new
    tokens of every sequence over [shared prefix | own cache | new tokens].

    q [B, T, heads_q, D] bf16 (strides between sequences and tokens free, as in
    a view of a fused projection), D 64 or 128; k_cache, v_cache [B, max_len,
    heads_kv, D], bf16, or float8_e4m3fn with k_scale, v_scale uint8 [B,
    max_len, heads_kv]; cache_len int32 [B].  k_new, v_new [B, T, heads_kv, D]
    bf16 are the new tokens' own entries: token t sees itself and its ancestors
    by ``parent`` (int32 [B, T], parent[b][0] = -1, as tree_run's; None: a
    chain); without them the queries see the cache (and prefix) only.
    k_prefix, v_prefix [prefix_len, heads_kv, D] of the cache's type, with
    their scales, are one copy for the whole batch.  ``scale`` (default
    1/sqrt(D)) multiplies the products.  ``lse`` float32 [B, T, heads_q]
    receives the logarithms of the sums, ``status`` int32 [1] the SV_ATTN_*
    bits.  Returns out [B, T, heads_q, D] bf16; enqueues on the current torch
    stream (or ``stream``) and does not synchronise."""
    import torch
    dev = q.get_device()
    if q.dim() != 4 or k_cache.dim() != 4 or dev < 0:
        raise ValueError("q must be a CUDA tensor [B, T, heads_q, head_dim], the caches [B, max_len, heads_kv, head_dim]")
    B, T, Hq, D = q.shape
    _, L, H, _ = k_cache.shape
    qb, qt = _tokens("q", q, q.shape, dev)
    if k_cache.shape != (B, L, H, D) or v_cache.shape != (B, L, H, D) or v_cache.dtype is not k_cache.dtype \
            or k_cache.get_device() != dev or v_cache.get_device() != dev or not k_cache.is_contiguous() \
            or not v_cache.is_contiguous():
        raise ValueError(f"k_cache and v_cache must be contiguous [{B}, max_len, heads_kv, {D}] of one type")
    fmt = _kv_format(k_cache, k_scale, "k_cache")
    _kv_format(v_cache, v_scale, "v_cache")
    _int32("cache_len", cache_len, (B,), dev)
    if (k_new is None) != (v_new is None) or (k_prefix is None) != (v_prefix is None):
        raise ValueError("keys and values come together")
    nb = nt = kn = vn = par = kp = vp = Lp = 0
    if k_new is not None:
        nb, nt = _tokens("k_new", k_new, (B, T, H, D), dev)
        if _tokens("v_new", v_new, (B, T, H, D), dev) != (nb, nt):
            raise ValueError("k_new and v_new must have the same strides")
        kn, vn = k_new.data_ptr(), v_new.data_ptr()
        if parent is not None:
            _int32("parent", parent, (B, T), dev)
            par = parent.data_ptr()
    elif parent is not None:
        raise ValueError("parent goes with k_new and v_new")
    if k_prefix is not None:
        Lp = k_prefix.shape[0]
        for name, t, ts in (("k_prefix", k_prefix, k_prefix_scale), ("v_prefix", v_prefix, v_prefix_scale)):
            if t.shape != (Lp, H, D) or t.dtype is not k_cache.dtype or t.get_device() != dev or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous [prefix_len, {H}, {D}] of the cache's type")
            _kv_format(t, ts, name)
        kp, vp = k_prefix.data_ptr(), v_prefix.data_ptr()
    elif k_prefix_scale is not None or v_prefix_scale is not None:
        raise ValueError("prefix scales go with a prefix")
    if out is not None and (out.shape != q.shape or out.dtype is not torch.bfloat16 or not out.is_contiguous()
                            or out.get_device() != dev):
        raise ValueError("out must be contiguous bfloat16 of q's shape")
    if lse is not None and (lse.shape != (B, T, Hq) or lse.dtype is not torch.float32 or not lse.is_contiguous()
                            or lse.get_device() != dev):
        raise ValueError("lse must be contiguous float32 [B, T, heads_q]")
    if status is not None:
        _int32("status", status, (1,), dev)
    nbytes = _attention_bytes(B, T, Hq, H, D, L, Lp, fmt)
    # the workspace comes from the caching allocator, for this call alone: calls on
    # other streams and captured graphs each have their own
    if stream is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        if out is None:
            out = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device=q.device)
    else:
        with torch.cuda.stream(stream):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
            if out is None:
                out = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device=q.device)
    args = _ATTENTION_ARGS.pack(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), 0 if k_scale is None else k_scale.data_ptr(),
        0 if v_scale is None else v_scale.data_ptr(), cache_len.data_ptr(), kp, vp,
        0 if k_prefix_scale is None else k_prefix_scale.data_ptr(),
        0 if v_prefix_scale is None else v_prefix_scale.data_ptr(), kn, vn, par, out.data_ptr(),
        0 if lse is None else lse.data_ptr(), 0 if status is None else status.data_ptr(), ws.data_ptr(), nbytes, qb, qt,
        nb, nt, B, T, Hq, H, D, L, Lp, fmt, D ** -0.5 if scale is None else scale)
    st = _on(dev, spec_verify_attention, args, _raw_stream(dev, stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_attention")
    return out


def lm_head_logits(hidden, weight, out=None, stream=None):
    """logits = hidden @ weight.T on the tensor cores (bf16 in, f32 out);
    hidden [M, K] and weight [V, K] contiguous bf16 CUDA tensors."""
    import torch
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16 or hidden.dim() != 2 or weight.dim() != 2 \
            or hidden.shape[1] != weight.shape[1] or not hidden.is_contiguous() or not weight.is_contiguous():
        raise ValueError("hidden [M, K] and weight [V, K] must be contiguous bf16")
    M, K = hidden.shape
    V = weight.shape[0]
    if out is None:
        out = torch.empty((M, V), dtype=torch.float32, device=hidden.device)
    s = stream if stream is not None else torch.cuda.current_stream(hidden.device)
    st = load().spec_verify_lm_head_logits(_ptr(hidden), _ptr(weight), M, V, K, _ptr(out), s.cuda_stream)
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_lm_head_logits")
    return out


def selftest_timeout(limit_us: int = 10000, stream=None) -> bool:
    """True when a kernel wait that nothing satisfies gave up within
    limit_us and reported it (the library's bounded-wait failure detection)."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    flag = _I(0)
    st = load().spec_verify_selftest_timeout(int(limit_us), ctypes.byref(flag), s.cuda_stream)
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_selftest_timeout")
    return bool(flag.value)
