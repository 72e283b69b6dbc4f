"""Thin ctypes binding over the C ABI in ``include/spec_verify.h``.

Argument marshalling only: every step of the verify path runs in the CUDA kernels of
``libspecverify.so``.  PyTorch supplies device memory and the current stream.  There is no CPU
fallback: if the library is missing or a call fails, these functions raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

from . import build_ext

SPEC_F32, SPEC_BF16, SPEC_F16 = 0, 1, 2
ROW_OK, ROW_NONFINITE, ROW_DEGENERATE, ROW_BAD_TOKEN, ROW_TIMEOUT = 0, 1, 2, 3, 4
ROW_BAD_PARENT, ROW_OVERFLOW, ROW_BAD_UNIFORM, ROW_BAD_QROW = 5, 6, 7, 8
ROW_BAD_PAGE, ROW_BAD_LENGTH, ROW_BAD_NODE, ROW_NO_PAGES, ROW_BAD_PARAM = 9, 10, 11, 12, 13

# every symbol the header declares
EXPORTS = ("spec_workspace_bytes", "spec_verify", "spec_verify_topk", "spec_verify_topp",
           "spec_verify_masked",
           "tree_verify_greedy", "spec_verify_greedy",
           "tree_verify_sample", "tree_verify_typical", "smc_verify", "spec_verify_noalloc", "spec_set_kernel_events", "spec_set_wait_limit",
           "spec_set_tree_sample_cluster", "spec_status_string",
           "process_logits", "kv_cache_write", "kv_cache_read", "verify_attention",
           "verify_attention_workspace_bytes", "qk_norm_rope", "kv_pages_reserve", "kv_pages_release",
           "sample_logits", "verify_attention_window")

# fixed scratch of spec_verify_noalloc (SPEC_NOALLOC_SCRATCH_BYTES in the header)
NOALLOC_SCRATCH_BYTES = 8 << 20
SPEC_ERR_TOO_LARGE = 4

_lib = None


class SpecVerifyError(RuntimeError):
    pass


def load(path: str | None = None):
    """Load the compiled library (building it first if the sources are newer)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or build_ext.LIB
    if not os.path.exists(path):
        raise SpecVerifyError(
            f"CUDA extension {path} is missing; build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.spec_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.spec_workspace_bytes.restype = Z
    lib.spec_verify.argtypes = [P, P, I, P, P, I, I, I, F, P, P, P, P, P, P, P, Z, P]
    lib.spec_verify.restype = I
    lib.spec_verify_topk.argtypes = [P, P, I, P, P, I, I, I, F, I, P, P, P, P, P, P, P, Z, P]
    lib.spec_verify_topk.restype = I
    lib.spec_verify_topp.argtypes = [P, P, I, P, P, I, I, I, F, F, P, P, P, P, P, P, P, Z, P]
    lib.spec_verify_topp.restype = I
    lib.spec_verify_masked.argtypes = [P, P, I, P, P, P, I, I, I, F, P, P, P, P, P, P, P, Z, P]
    lib.spec_verify_masked.restype = I
    lib.tree_verify_greedy.argtypes = [P, I, P, P, I, I, I, I, P, P, P, P, P, Z, P]
    lib.tree_verify_greedy.restype = I
    lib.spec_verify_greedy.argtypes = [P, I, P, I, I, I, P, P, P, P, Z, P]
    lib.spec_verify_greedy.restype = I
    lib.tree_verify_sample.argtypes = [P, P, I, P, P, P, P, I, I, I, I, F, I, P, P, P, P, P, P]
    lib.tree_verify_sample.restype = I
    lib.tree_verify_typical.argtypes = [P, I, P, P, P, I, I, I, F, F, F, I, P, P, P, P, P, P, P, Z, P]
    lib.tree_verify_typical.restype = I
    lib.smc_verify.argtypes = [P, P, I, P, P, P, I, I, I, I, F, F, P, P, P, P, P, P, P, P, P, Z, P]
    lib.smc_verify.restype = I
    lib.spec_verify_noalloc.argtypes = [P, P, I, P, P, I, I, I, F, P, P, P, P, P, P, P]
    lib.spec_verify_noalloc.restype = I
    lib.process_logits.argtypes = [P, P, I, I, I, I, P, P, P, P, I, P, I, P, P, P, P, P, P, P, I, P, P, P]
    lib.process_logits.restype = I
    lib.kv_cache_write.argtypes = [P, P, P, P, I, I, I, I, I, P, P, P, P, I, I, P, I, P, P, P, I, P, P, P]
    lib.kv_cache_write.restype = I
    lib.kv_cache_read.argtypes = [P, P, P, P, I, I, I, I, P, I, P, P, I, I, P, P, I, P, P]
    lib.kv_cache_read.restype = I
    lib.verify_attention.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, P, I, I, P, I, P, P, P, F,
                                     P, P, P, P, Z, P]
    lib.verify_attention.restype = I
    lib.verify_attention_window.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, P, I, I, P, I, P, P, P, I, I, F,
                                            P, P, P, P, Z, P]
    lib.verify_attention_window.restype = I
    lib.verify_attention_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.verify_attention_workspace_bytes.restype = Z
    lib.qk_norm_rope.argtypes = [P, P, P, P, I, I, I, I, I, I, P, P, I, F, P, I, I, I, P, P, P, P, P, P, P, P, P]
    lib.qk_norm_rope.restype = I
    lib.kv_pages_reserve.argtypes = [P, I, P, P, P, I, I, I, P, I, P, P, P, P]
    lib.kv_pages_reserve.restype = I
    lib.kv_pages_release.argtypes = [P, I, P, P, I, I, P, I, P, P, P]
    lib.kv_pages_release.restype = I
    lib.sample_logits.argtypes = [P, ctypes.c_int64, I, I, I, P, P, P, P, P, P, P, P, P]
    lib.sample_logits.restype = I
    lib.spec_set_kernel_events.argtypes = [P, P]
    lib.spec_set_kernel_events.restype = None
    lib.spec_set_wait_limit.argtypes = [I]
    lib.spec_set_wait_limit.restype = I
    lib.spec_set_tree_sample_cluster.argtypes = [I]
    lib.spec_set_tree_sample_cluster.restype = I
    lib.spec_status_string.argtypes = [I]
    lib.spec_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int):
    if rc != 0:
        raise SpecVerifyError(load().spec_status_string(rc).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype in (torch.bfloat16, torch.int16):  # int16 = raw bf16 bit patterns
        return SPEC_BF16
    raise TypeError(f"logits must be bfloat16 (or its int16 bits) or float32, got {t.dtype}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise SpecVerifyError("verify inputs must be CUDA tensors (there is no CPU path)")


class Workspace:
    """Device scratch for the verify calls, grown on demand (plain torch allocation)."""

    def __init__(self, device=None):
        self.device = torch.device(device or "cuda")
        self.buf = None

    def get(self, nbytes: int) -> torch.Tensor:
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        return self.buf


_default_ws = {}


def _workspace(ws, device):
    if ws is not None:
        return ws
    key = str(device)
    if key not in _default_ws:
        _default_ws[key] = Workspace(device)
    return _default_ws[key]


def set_kernel_events(start=None, stop=None):
    """Time the dominant kernel of later calls: torch.cuda.Event pair (recorded around it on the
    call's stream), or None to stop."""
    if start is None or stop is None:
        load().spec_set_kernel_events(None, None)
        return
    for e in (start, stop):
        if not e.cuda_event:
            e.record()  # creates the underlying CUDA event
    load().spec_set_kernel_events(ctypes.c_void_p(start.cuda_event), ctypes.c_void_p(stop.cuda_event))


def set_wait_limit(polls: int) -> int:
    """Test aid: polls after which a bounded wait of the streaming kernels gives up (0: at once,
    so every request of a streaming call reports ROW_TIMEOUT; negative: the default).  Returns
    the previous limit."""
    return int(load().spec_set_wait_limit(int(polls)))


def set_tree_sample_cluster(cl: int) -> int:
    """Measurement aid: force tree_verify_sample's cluster size (1, 2, 4, 8 or 16 CTAs per request;
    anything else: the automatic choice).  Returns the previous setting (0: automatic)."""
    return int(load().spec_set_tree_sample_cluster(int(cl)))


def workspace_bytes(B, gamma, V, top_k=0, tree_nodes=0) -> int:
    return int(load().spec_workspace_bytes(B, gamma, V, top_k, tree_nodes))


def spec_verify(target, draft, draft_tokens, uniforms, temperature: float, *, top_k: int = 0,
                allowed=None, top_p: float | None = None, aux: bool = False, out=None,
                workspace: Workspace | None = None, stream=None):
    """Exact speculative-sampling verify on the GPU.

    target [B, gamma+1, V], draft [B, gamma, V] (bf16 / int16 bf16 bits / fp32, CUDA),
    draft_tokens [B, gamma] int32, uniforms [B, gamma+2] fp32.  ``top_k`` > 0 applies the top-k
    processor (spec_verify_topk).  ``allowed`` (CUDA int32/uint32 [B, gamma+1, ceil(V/32)]) is a
    grammar mask (spec_verify_masked; not with top_k); ``top_p`` applies the top-p processor
    (spec_verify_topp; alone).  Returns a dict of CUDA tensors:
    accepted_len, out_tokens, row_status (and lse_p, lse_q, accept when ``aux``).
    """
    lib = load()
    _need_cuda(target, draft, draft_tokens, uniforms)
    B, g1, V = target.shape
    gamma = g1 - 1
    dev = target.device
    if out is None:
        out = dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            out_tokens=torch.empty(B, gamma + 1, dtype=torch.int32, device=dev),
            row_status=torch.empty(B, dtype=torch.int32, device=dev),
        )
        if aux:
            out["lse_p"] = torch.empty(B, gamma + 1, dtype=torch.float32, device=dev)
            out["lse_q"] = torch.empty(B, gamma, dtype=torch.float32, device=dev)
            out["accept"] = torch.empty(B, gamma, dtype=torch.float32, device=dev)
    nbytes = workspace_bytes(B, gamma, V, top_k)
    ws = _workspace(workspace, dev).get(nbytes)
    common = [_ptr(target), _ptr(draft), _dtype_code(target), _ptr(draft_tokens), _ptr(uniforms),
              B, gamma, V, float(temperature)]
    tail = [_ptr(out["accepted_len"]), _ptr(out["out_tokens"]), _ptr(out.get("row_status")),
            _ptr(out.get("lse_p")), _ptr(out.get("lse_q")), _ptr(out.get("accept")),
            _ptr(ws), ws.numel(), _stream(stream)]
    if top_p is not None:
        if top_k or allowed is not None:
            raise ValueError("spec_verify_topp takes no top_k or mask")
        rc = lib.spec_verify_topp(*common, float(top_p), *tail)
    elif allowed is not None:
        if top_k:
            raise ValueError("spec_verify_masked takes no top_k")
        _need_cuda(allowed)
        W = (V + 31) // 32
        if tuple(allowed.shape) != (B, gamma + 1, W) or allowed.element_size() != 4 \
                or not allowed.is_contiguous():
            raise ValueError(f"allowed must be a contiguous 32-bit [B, gamma+1, {W}] tensor")
        rc = lib.spec_verify_masked(*common[:5], _ptr(allowed), *common[5:], *tail)
    elif top_k:
        rc = lib.spec_verify_topk(*common, int(top_k), *tail)
    else:
        rc = lib.spec_verify(*common, *tail)
    _check(rc)
    return out


def spec_verify_topp(target, draft, draft_tokens, uniforms, temperature: float, top_p: float, **kw):
    """spec_verify with the top-p (nucleus) processor on every row."""
    return spec_verify(target, draft, draft_tokens, uniforms, temperature, top_p=top_p, **kw)


def spec_verify_masked(target, draft, draft_tokens, uniforms, allowed, temperature: float, **kw):
    """spec_verify under a grammar mask ``allowed`` [B, gamma+1, ceil(V/32)] (32-bit words)."""
    return spec_verify(target, draft, draft_tokens, uniforms, temperature, allowed=allowed, **kw)


def spec_verify_noalloc(target, draft, draft_tokens, uniforms, temperature: float, *,
                        aux: bool = False, out=None, stream=None):
    """spec_verify through the entry point that allocates no device scratch.

    For callers that cannot allocate device memory: the library keeps the scratch in a fixed
    per-GPU array of NOALLOC_SCRATCH_BYTES, shared by every call on that GPU, so calls must not
    overlap on the GPU.  Pass ``out`` (preallocated CUDA tensors, same keys as spec_verify's
    result) to keep this wrapper itself from allocating.  Sizes that need more scratch than the
    array holds raise SpecVerifyError.
    """
    lib = load()
    _need_cuda(target, draft, draft_tokens, uniforms)
    B, g1, V = target.shape
    gamma = g1 - 1
    dev = target.device
    if out is None:
        out = dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            out_tokens=torch.empty(B, gamma + 1, dtype=torch.int32, device=dev),
            row_status=torch.empty(B, dtype=torch.int32, device=dev),
        )
        if aux:
            out["lse_p"] = torch.empty(B, gamma + 1, dtype=torch.float32, device=dev)
            out["lse_q"] = torch.empty(B, gamma, dtype=torch.float32, device=dev)
            out["accept"] = torch.empty(B, gamma, dtype=torch.float32, device=dev)
    rc = lib.spec_verify_noalloc(
        _ptr(target), _ptr(draft), _dtype_code(target), _ptr(draft_tokens), _ptr(uniforms),
        B, gamma, V, float(temperature), _ptr(out["accepted_len"]), _ptr(out["out_tokens"]),
        _ptr(out.get("row_status")), _ptr(out.get("lse_p")), _ptr(out.get("lse_q")),
        _ptr(out.get("accept")), _stream(stream))
    _check(rc)
    return out


def spec_verify_topk(target, draft, draft_tokens, uniforms, temperature: float, top_k: int, **kw):
    if top_k < 1:
        raise ValueError("top_k must be >= 1")
    return spec_verify(target, draft, draft_tokens, uniforms, temperature, top_k=top_k, **kw)


def tree_verify_greedy(logits, parents, tokens, *, max_out: int | None = None, out=None,
                       workspace: Workspace | None = None, stream=None):
    """Greedy tree verify on the GPU.  logits [B, N+1, V]; parents, tokens [B, N] int32."""
    lib = load()
    _need_cuda(logits, parents, tokens)
    B, n1, V = logits.shape
    N = n1 - 1
    max_out = N + 1 if max_out is None else int(max_out)
    dev = logits.device
    if out is None:
        out = dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            out_tokens=torch.empty(B, max_out, dtype=torch.int32, device=dev),
            out_nodes=torch.empty(B, max(max_out - 1, 0), dtype=torch.int32, device=dev),
            row_status=torch.empty(B, dtype=torch.int32, device=dev),
        )
    nbytes = workspace_bytes(B, 0, V, 0, max(N, 1))
    ws = _workspace(workspace, dev).get(nbytes)
    rc = lib.tree_verify_greedy(_ptr(logits), _dtype_code(logits), _ptr(parents), _ptr(tokens),
                                B, N, V, max_out, _ptr(out["accepted_len"]),
                                _ptr(out["out_tokens"]), _ptr(out.get("out_nodes")),
                                _ptr(out.get("row_status")), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc)
    return out


def tree_verify_typical(logits, parents, tokens, uniforms, temperature: float, epsilon: float,
                        delta: float, *, max_out: int | None = None, aux: bool = False, out=None,
                        workspace: Workspace | None = None, stream=None):
    """Tree verify with typical acceptance on the GPU.  logits [B, N+1, V] (bf16 / int16 bf16
    bits / fp32, CUDA), parents and tokens [B, N] int32, uniforms [B] fp32.  Returns a dict of CUDA
    tensors: accepted_len, out_tokens [B, max_out], out_nodes, row_status (and entropy [B, N+1],
    logp [B, N] when ``aux``)."""
    lib = load()
    _need_cuda(logits, parents, tokens, uniforms)
    B, R, V = logits.shape
    N = R - 1
    mo = N + 1 if max_out is None else int(max_out)
    dev = logits.device
    if out is None:
        out = dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            out_tokens=torch.empty(B, mo, dtype=torch.int32, device=dev),
            out_nodes=torch.empty(B, max(mo - 1, 0), dtype=torch.int32, device=dev),
            row_status=torch.empty(B, dtype=torch.int32, device=dev),
        )
        if aux:
            out["entropy"] = torch.empty(B, R, dtype=torch.float32, device=dev)
            out["logp"] = torch.empty(B, N, dtype=torch.float32, device=dev)
    nbytes = workspace_bytes(B, 0, V, 0, max(N, 1))
    ws = _workspace(workspace, dev).get(nbytes)
    rc = lib.tree_verify_typical(
        _ptr(logits), _dtype_code(logits), _ptr(parents), _ptr(tokens), _ptr(uniforms), B, N, V,
        float(temperature), float(epsilon), float(delta), mo, _ptr(out["accepted_len"]),
        _ptr(out["out_tokens"]), _ptr(out.get("out_nodes")), _ptr(out.get("row_status")),
        _ptr(out.get("entropy")), _ptr(out.get("logp")), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc)
    return out


def tree_verify_sample(target, draft, parents, tokens, qrow, uniforms, temperature: float, *,
                       max_out: int | None = None, aux: bool = False, out=None, stream=None):
    """Stochastic tree verify on the GPU (residual update over each node's children).

    target [B, N+1, V], draft [B, Nq, V] (same dtype), parents / tokens / qrow [B, N] int32,
    uniforms [B, N+1] float32; all CUDA tensors.  Returns accepted_len, out_tokens, out_nodes,
    row_status and, with ``aux``, accept [B, N] (NaN where a node was not tested).
    """
    lib = load()
    _need_cuda(target, draft, parents, tokens, qrow, uniforms)
    B, n1, V = target.shape
    N = n1 - 1
    Nq = draft.shape[1] if draft is not None and draft.dim() == 3 else 0
    if draft is not None and N > 0 and (draft.shape[0] != B or draft.shape[2] != V or
                                        _dtype_code(draft) != _dtype_code(target)):
        raise ValueError("draft must be [B, Nq, V] with the target's dtype")
    max_out = N + 1 if max_out is None else int(max_out)
    dev = target.device
    if out is None:
        out = dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            out_tokens=torch.empty(B, max_out, dtype=torch.int32, device=dev),
            out_nodes=torch.empty(B, max(max_out - 1, 0), dtype=torch.int32, device=dev),
            row_status=torch.empty(B, dtype=torch.int32, device=dev),
        )
        if aux:
            out["accept"] = torch.empty(B, N, dtype=torch.float32, device=dev)
    rc = lib.tree_verify_sample(_ptr(target), _ptr(draft) if Nq > 0 else None, _dtype_code(target),
                                _ptr(parents), _ptr(tokens), _ptr(qrow), _ptr(uniforms), B, N, Nq,
                                V, float(temperature), max_out, _ptr(out["accepted_len"]),
                                _ptr(out["out_tokens"]), _ptr(out.get("out_nodes")),
                                _ptr(out.get("row_status")), _ptr(out.get("accept")),
                                _stream(stream))
    _check(rc)
    return out


def smc_verify(target, draft, draft_tokens, log_weights, uniforms, groups: int, temperature: float,
               ess_threshold: float, *, out=None, workspace: Workspace | None = None, stream=None):
    """The verify side of one SMC-SD round on the GPU.

    target [B, K+1, V], draft [B, K, V], draft_tokens [B, K] int32, log_weights [B] float32,
    uniforms [B, 2] float32, B = groups * particles.  Returns out_tokens, accepted_len, row_status,
    log_weights (after the round), block_log_ratio, ess, resampled and ancestors.
    """
    lib = load()
    _need_cuda(target, draft, draft_tokens, log_weights, uniforms)
    B, k1, V = target.shape
    K = k1 - 1
    if groups < 1 or B % groups:
        raise ValueError("the batch must split into equal groups of particles")
    Np = B // groups
    dev = target.device
    if out is None:
        out = dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            out_tokens=torch.empty(B, K + 1, dtype=torch.int32, device=dev),
            row_status=torch.empty(B, dtype=torch.int32, device=dev),
            log_weights=torch.empty(B, dtype=torch.float32, device=dev),
            block_log_ratio=torch.empty(B, dtype=torch.float32, device=dev),
            ess=torch.empty(groups, dtype=torch.float32, device=dev),
            resampled=torch.empty(groups, dtype=torch.int32, device=dev),
            ancestors=torch.empty(B, dtype=torch.int32, device=dev),
        )
    nbytes = workspace_bytes(B, K, V)
    ws = _workspace(workspace, dev).get(nbytes)
    rc = lib.smc_verify(_ptr(target), _ptr(draft) if K > 0 else None, _dtype_code(target),
                        _ptr(draft_tokens), _ptr(log_weights), _ptr(uniforms), groups, Np, K, V,
                        float(temperature), float(ess_threshold), _ptr(out["accepted_len"]),
                        _ptr(out["out_tokens"]), _ptr(out["log_weights"]),
                        _ptr(out.get("block_log_ratio")), _ptr(out.get("ess")),
                        _ptr(out.get("resampled")), _ptr(out.get("ancestors")),
                        _ptr(out.get("row_status")), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc)
    return out


def spec_verify_greedy(target, draft_tokens, *, out=None, workspace: Workspace | None = None,
                       stream=None):
    """Linear greedy verify on the GPU.  target [B, gamma+1, V]; draft_tokens [B, gamma] int32."""
    lib = load()
    _need_cuda(target, draft_tokens)
    B, g1, V = target.shape
    gamma = g1 - 1
    dev = target.device
    if out is None:
        out = dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            out_tokens=torch.empty(B, gamma + 1, dtype=torch.int32, device=dev),
            row_status=torch.empty(B, dtype=torch.int32, device=dev),
        )
    nbytes = workspace_bytes(B, 0, V, 0, max(gamma, 1))
    ws = _workspace(workspace, dev).get(nbytes)
    rc = lib.spec_verify_greedy(_ptr(target), _dtype_code(target), _ptr(draft_tokens), B, gamma, V,
                                _ptr(out["accepted_len"]), _ptr(out["out_tokens"]),
                                _ptr(out.get("row_status")), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc)
    return out


# ------------------------------------------------------------------ around the verify step

class KVCache(NamedTuple):
    """The 8-bit paged cache: e4m3 codes [pages, heads, page_size, head_dim] of keys and values, and one fp32
    scale, a power of two, per page and head.  The calls take any four such tensors in this order."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def kv_cache(pages: int, heads: int, page_size: int, head_dim: int, device="cuda") -> KVCache:
    """An empty cache (page_size 16, 32, 64 or 128; head_dim 64 or 128)."""
    shape = (pages, heads, page_size, head_dim)
    return KVCache(*(torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)),
                   *(torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2)))


# With `stream` a call runs there instead of on the current stream: the caller orders it after the work on its inputs, and keeps
# them until it has run.
#
# A round's calls are short and many, so their marshalling avoids what costs microseconds: pointers go as plain ints,
# dense tensors pass no strides, and the current stream's handle comes without a Stream object.

_EMPTY = torch.empty


def _new(shape, dtype, device, stream):
    """A new tensor for a call on `stream`.  It is allocated on that stream: a block freed on the current one may still be in
    use there.  The current stream, where the caller goes on, is noted as its second user."""
    if stream is None:
        # (torch takes sizes one by one in two thirds of a tuple's time)
        return _EMPTY(shape, dtype=dtype, device=device) if type(shape) is int else _EMPTY(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = _EMPTY(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


_EMPTY_LIKE, _DENSE = torch.empty_like, torch.contiguous_format


def _like(t, stream):
    """As _new, contiguous and with t's shape, dtype and device (which takes half the time)."""
    if stream is None:
        return _EMPTY_LIKE(t, memory_format=_DENSE)
    return _new(t.shape, t.dtype, t.device, stream)


def _raw_stream(stream, at) -> int:
    if stream is not None:
        if stream.device_index != at:
            raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors on cuda:{at}")
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(at)


def _capturing(stream) -> bool:
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


_round_ws = {}


def _round_workspace(ws, device, stream, raw, nbytes):
    """The call's workspace; by default one per device and stream, as calls on two streams may overlap.  A captured call has one
    of its own, from its graph's memory: graphs captured on one stream may be replayed on two, and a kept workspace may be
    replaced by a larger one."""
    if ws is not None:
        return ws.get(nbytes)
    if _capturing(stream):
        return _new(nbytes, torch.uint8, device, stream)
    key = (device, raw)
    buf = _round_ws.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = _round_ws[key] = _new(nbytes, torch.uint8, device, stream)
    return buf


_ROUND_DTYPES = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}


def _round_dtype(dtype, what: str, allowed) -> int:
    code = _ROUND_DTYPES.get(dtype)
    if code not in allowed:
        raise TypeError(f"{what} has an unsupported dtype {dtype}")
    return code


def _strides(t, n):
    """The strides of the n leading dimensions for the C ABI (None: dense); the last one must be contiguous.  A dimension
    of size 1 has no stride that matters, and torch may give it any."""
    if t.is_contiguous():
        return None
    shape, st = t.shape, t.stride()
    kept = _kept_strides.get((shape, st, n))
    if kept is not None:
        return kept
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError("the last dimension must be contiguous")
    key = (shape, st, n)
    if 1 in shape[:n]:
        dense = [1] * t.dim()
        for i in range(t.dim() - 2, -1, -1):
            dense[i] = dense[i + 1] * shape[i + 1]
        st = [s if m > 1 else d for s, m, d in zip(st, shape, dense)]
    if len(_kept_strides) >= 1024:  # shapes that change without end
        _kept_strides.clear()
    kept = _kept_strides[key] = _STRIDES[n](*st[:n])
    return kept


_kept_strides = {}  # what the C ABI only reads, by shape and strides
_STRIDES = {n: ctypes.c_int64 * n for n in (2, 3)}


def _not_at(t, at):
    if t.get_device() < 0:
        raise SpecVerifyError("the tensors of a call must be CUDA tensors (there is no CPU path)")
    raise ValueError(f"a tensor is on cuda:{t.get_device()}, the others on cuda:{at}")


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _at(t) -> int:
    """The device of a call, which launches on the current one."""
    at = t.get_device()
    if at < 0:
        _not_at(t, at)
    if at != _current_device():
        raise ValueError(f"the tensors are on cuda:{at}, the current device is cuda:{_current_device()}")
    return at


def _arg(t, dtype, shape, what, at):
    """The pointer of an optional argument: a contiguous tensor of this dtype and shape on device `at`."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    if t.get_device() != at:
        _not_at(t, at)
    return t.data_ptr()


_I32, _F32 = torch.int32, torch.float32


def _int(x, what):
    """A whole number for the C ABI's int, which would drop the bits above 32 without a word."""
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{what} is out of range: {x}")
    return x


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _cache_args(cache, page_table, lens, B, at):
    k, v, ks, vs = cache
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("the cache's codes must be contiguous [pages, heads, page_size, head_dim]")
    if k.dtype not in _CODES or v.dtype not in _CODES:
        raise TypeError("the cache's codes must be float8_e4m3fn (or their bytes as uint8)")
    for t in (k, v):
        if t.get_device() != at:
            _not_at(t, at)
    pages, heads, page, dim = shape
    if page_table is None or page_table.dim() != 2 or page_table.shape[0] != B or lens is None:
        raise ValueError(f"page_table must be [{B}, width], with lens [{B}]")
    width = page_table.shape[1]
    scales = (pages, heads)
    return (pages, heads, page, dim, width,
            (k.data_ptr(), v.data_ptr(), _arg(ks, _F32, scales, "k_scale", at), _arg(vs, _F32, scales, "v_scale", at)),
            _arg(page_table, _I32, (B, width), "page_table", at), _arg(lens, _I32, (B,), "lens", at))


def process_logits(logits, *, tokens=None, parents=None, history=None, prompt_len=None, history_len=None,
                   repetition=None, presence=None, frequency=None, bias_tokens=None, bias_values=None,
                   allowed=None, out=None, stream=None):
    """Penalties for repeated tokens, biases and a grammar mask on the rows of a round.

    logits [B, R, V] (bf16 or fp32, CUDA; any request and row stride).  Row r follows the drafted ``tokens``
    [B, N] on its path: tokens 0..r-1, or, with ``parents`` [B, N], node r-1 and its ancestors (R <= N + 1).
    ``history`` [B, H]: the tokens before the round, ``history_len`` [B] of them valid, the first
    ``prompt_len`` [B] the prompt (which counts for the repetition penalty alone).  ``repetition``, ``presence``,
    ``frequency`` [B] float32; ``bias_tokens`` / ``bias_values`` [B, nb]; ``allowed`` [B, R, ceil(V/32)] 32-bit
    words as in spec_verify_masked.  ``out`` = dict(logits=..., row_status=...); out["logits"] may be ``logits``.
    Returns that dict.
    """
    lib = load()
    at = _at(logits)
    if logits.dim() != 3:
        raise ValueError("logits must be [B, R, V]")
    B, R, V = logits.shape
    dev = logits.device
    dt = _round_dtype(logits.dtype, "logits", (SPEC_F32, SPEC_BF16))
    N = 0 if tokens is None else tokens.shape[-1]
    H = 0 if history is None else history.shape[-1]
    nb = 0 if bias_tokens is None else bias_tokens.shape[-1]
    if nb and bias_values is None:
        raise ValueError("bias_tokens need bias_values")
    if parents is not None and tokens is None:
        raise ValueError("parents need tokens")
    if R > N + 1:
        raise ValueError(f"{R} rows need at least {R - 1} drafted tokens")
    if out is None:
        y = _new((B, R, V), logits.dtype, dev, stream)
        out = {"logits": y, "row_status": _new(B, _I32, dev, stream)}
    else:
        y = out["logits"]
        if y.shape != logits.shape or y.dtype is not logits.dtype:
            raise ValueError("out['logits'] must have the logits' shape and dtype")
        if y.get_device() != at:
            _not_at(y, at)
    if allowed is not None:
        W = (V + 31) // 32
        if allowed.get_device() != at:
            _not_at(allowed, at)
        if tuple(allowed.shape) != (B, R, W) or allowed.element_size() != 4 or not allowed.is_contiguous():
            raise ValueError(f"allowed must be a contiguous 32-bit [B, R, {W}] tensor")
    one = (B,)
    rc = lib.process_logits(
        logits.data_ptr(), y.data_ptr(), dt, B, R, V, _strides(logits, 2), _strides(y, 2),
        _arg(tokens, _I32, (B, N), "tokens", at) if N else None, _arg(parents, _I32, (B, N), "parents", at) if N else None, N,
        _arg(history, _I32, (B, H), "history", at) if H else None, H, _arg(prompt_len, _I32, one, "prompt_len", at),
        _arg(history_len, _I32, one, "history_len", at), _arg(repetition, _F32, one, "repetition", at),
        _arg(presence, _F32, one, "presence", at), _arg(frequency, _F32, one, "frequency", at),
        _arg(bias_tokens, _I32, (B, nb), "bias_tokens", at) if nb else None,
        _arg(bias_values, _F32, (B, nb), "bias_values", at) if nb else None, nb,
        None if allowed is None else allowed.data_ptr(), _arg(out.get("row_status"), _I32, one, "row_status", at),
        _raw_stream(stream, at))
    if rc:
        _check(rc)
    return out


def kv_cache_write(k, v, cache, page_table, lens, *, accepted_len=None, out_nodes=None, out=None, stream=None):
    """Appends rows to the requests' 8-bit caches, one scale per page and head.

    k, v [B, T, Hkv, D] (fp32, bf16 or fp16; any strides but the last), ``cache`` a KVCache (written in place),
    page_table [B, width] and lens [B] int32.  ``accepted_len`` [B] and ``out_nodes`` [B, width], as a verify call
    returns them, choose the rows: 0 .. accepted_len, or row 0 and the accepted path's nodes; without them
    all T rows are written.  Returns dict(lens, row_status): the lengths after the write.
    """
    lib = load()
    at = _at(k)
    if v.get_device() != at:
        _not_at(v, at)
    if k.dim() != 4 or k.shape != v.shape or k.dtype is not v.dtype:
        raise ValueError("k and v must be [B, T, heads, head_dim] of one dtype")
    B, T, heads, dim = k.shape
    dev = k.device
    dt = _round_dtype(k.dtype, "k", (SPEC_F32, SPEC_BF16, SPEC_F16))
    pages, h, page, d, width, ptrs, table, ln = _cache_args(cache, page_table, lens, B, at)
    if h != heads or d != dim:
        raise ValueError(f"the cache holds {h} heads of {d}, the rows {heads} of {dim}")
    if out_nodes is not None and accepted_len is None:
        raise ValueError("out_nodes need accepted_len")
    nw = 0 if out_nodes is None else out_nodes.shape[-1]
    if out is None:
        out = {"lens": _new(B, _I32, dev, stream), "row_status": _new(B, _I32, dev, stream)}
    one = (B,)
    acc, nodes = _arg(accepted_len, _I32, one, "accepted_len", at), _arg(out_nodes, _I32, (B, nw), "out_nodes", at)
    if out_nodes is not None and not nw:
        nodes = acc  # no node is read; a null pointer would say that the rows are a chain's
    rc = lib.kv_cache_write(
        k.data_ptr(), _strides(k, 3), v.data_ptr(), _strides(v, 3), dt, B, T, heads, dim, *ptrs, pages, page, table, width,
        ln, acc, nodes, nw, _arg(out.get("lens"), _I32, one, "lens", at),
        _arg(out.get("row_status"), _I32, one, "row_status", at), _raw_stream(stream, at))
    if rc:
        _check(rc)
    return out


def kv_cache_read(cache, page_table, lens, *, max_len: int, start=None, dtype=torch.bfloat16, out=None, stream=None):
    """Reads tokens start .. start + max_len - 1 of every request back as ``dtype``: dict(k, v [B, max_len, heads,
    head_dim], row_status).  Tokens past a request's length read as zero."""
    lib = load()
    B = lens.shape[0]
    at = _at(cache[0])
    pages, heads, page, dim, width, ptrs, table, ln = _cache_args(cache, page_table, lens, B, at)
    dev = cache[0].device
    shape = (B, max_len, heads, dim)
    if out is None:
        out = {"k": _new(shape, dtype, dev, stream), "v": _new(shape, dtype, dev, stream),
               "row_status": _new(B, _I32, dev, stream)}
    y, z = out["k"], out["v"]
    dt = _round_dtype(y.dtype, "out", (SPEC_F32, SPEC_BF16, SPEC_F16))
    one = (B,)
    rc = lib.kv_cache_read(*ptrs, pages, page, heads, dim, table, width, ln, _arg(start, _I32, one, "start", at), B, max_len,
                           _arg(y, y.dtype, shape, "out['k']", at), _arg(z, y.dtype, shape, "out['v']", at), dt,
                           _arg(out.get("row_status"), _I32, one, "row_status", at), _raw_stream(stream, at))
    if rc:
        _check(rc)
    return out


_attn_bytes = {}


def verify_attention(q, cache, page_table, lens, *, k=None, v=None, parents=None, n_rows=None,
                     scale: float | None = None, lse: bool = False, out=None, workspace: Workspace | None = None,
                     stream=None):
    """Attention of a round's rows over the 8-bit cache and the round's own keys and values.

    q [B, T, Hq, D] and k, v [B, T, Hkv, D] (bf16 or fp16; any strides but the last), T <= 256, Hq a multiple of
    Hkv; without k and v the rows see the cache alone.  Every row sees the committed tokens; of the round's rows, row t sees
    0..t, or with ``parents`` [B, T-1] (as the tree calls take it) row 0, its ancestors and itself.  ``n_rows`` [B]:
    live rows of each request.  ``scale`` defaults to D ** -0.5.  Returns dict(out [B, T, Hq, D], row_status and,
    with ``lse``, lse [B, T, Hq] in fp32).
    """
    return _attention(q, cache, page_table, lens, k, v, parents, n_rows, None, scale, lse, out, workspace, stream)


def verify_attention_window(q, cache, page_table, lens, *, window: int, sinks: int = 0, k, v, parents=None, n_rows=None,
                            scale: float | None = None, lse: bool = False, out=None, workspace: Workspace | None = None,
                            stream=None):
    """verify_attention under a sliding window: a row at position p (lens[b] plus its depth in the round) sees the tokens j with
    p - j < ``window``, and those with j < ``sinks``; of the round's rows those of its path that this leaves it.  Pages without
    a token that any row sees are not read: their entries in the table may be anything.  (kv_pages_release gives back a request's last
    pages, not those that have left a window.)  Arguments and result as there."""
    reach = (_int(window, "window"), _int(sinks, "sinks"))
    return _attention(q, cache, page_table, lens, k, v, parents, n_rows, reach, scale, lse, out, workspace, stream)


def _attention(q, cache, page_table, lens, k, v, parents, n_rows, window, scale, lse, out, workspace, stream):
    lib = load()
    at = _at(q)
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D]")
    shape = q.shape
    B, T, hq, dim = shape
    dev = q.device
    dt = _round_dtype(q.dtype, "q", (SPEC_BF16, SPEC_F16))
    pages, hkv, page, d, width, ptrs, table, ln = _cache_args(cache, page_table, lens, B, at)
    if d != dim or hq % hkv:
        raise ValueError(f"q has {hq} heads of {dim}, the cache {hkv} of {d}")
    if k is None and v is None:
        kp = vp = kst = vst = None
    elif k is None or v is None:
        raise ValueError("k and v come together")
    else:
        if k.shape != (B, T, hkv, dim) or v.shape != k.shape or k.dtype is not q.dtype or v.dtype is not q.dtype:
            raise ValueError("k and v must be [B, T, Hkv, D] of q's dtype")
        for t in (k, v):
            if t.get_device() != at:
                _not_at(t, at)
        kp, vp, kst, vst = k.data_ptr(), v.data_ptr(), _strides(k, 3), _strides(v, 3)
    if out is None:
        y = _like(q, stream)
        out = {"out": y, "row_status": _like(lens, stream)}
        if lse:
            out["lse"] = _new((B, T, hq), _F32, dev, stream)
    else:
        y = out["out"]
        if y.shape != shape or y.dtype is not q.dtype or not y.is_contiguous():
            raise ValueError("out['out'] must be contiguous, with q's shape and dtype")
        if y.get_device() != at:
            _not_at(y, at)
    key = (T, hq, hkv, dim)
    nbytes = _attn_bytes.get(key)
    if nbytes is None:
        nbytes = _attn_bytes[key] = int(lib.verify_attention_workspace_bytes(1, *key))
    raw = _raw_stream(stream, at)
    ws = _round_workspace(workspace, dev, stream, raw, max(nbytes, 256))
    if ws.get_device() != at:
        _not_at(ws, at)
    rc = (lib.verify_attention if window is None else lib.verify_attention_window)(
        q.data_ptr(), _strides(q, 3), kp, kst, vp, vst, dt, B, T, hq, hkv, dim, *ptrs, pages, page, table, width, ln,
        _arg(parents, _I32, (B, T - 1), "parents", at) if T > 1 else None, _arg(n_rows, _I32, (B,), "n_rows", at),
        *(window or ()), dim ** -0.5 if scale is None else scale, y.data_ptr(), _arg(out.get("lse"), _F32, (B, T, hq), "lse", at),
        _arg(out.get("row_status"), _I32, (B,), "row_status", at), ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc)
    return out


def rope_table(positions: int, dim: int, *, base: float = 10000.0, scale: float = 1.0, device="cuda"):
    """The table of qk_norm_rope, [positions, dim] in fp32: a position's dim / 2 cosines, then its sines, of the angles
    position * scale * base ** (-2 i / dim).  The angles are formed in 64 bits.  Made once a model."""
    if dim % 2 or dim < 2 or positions < 1:
        raise ValueError("a table needs positions and an even dim")
    inv = base ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim) * scale
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).to(_F32)


def qk_norm_rope(q, k, lens, rope, *, q_weight=None, k_weight=None, eps: float = 1e-6, parents=None, n_rows=None,
                 interleaved: bool = False, out=None, stream=None):
    """The round's queries and keys, each head normalised and rotated by its position, in one pass.

    q [B, T, Hq, D] and k [B, T, Hkv, D] (bf16 or fp16; any strides but the last, so views of one projection's output
    will do).  ``q_weight`` and ``k_weight`` [D] (the rows' dtype or fp32): the RMS norms' weights; without them there is
    no norm.  ``rope`` [positions, rot] fp32 as rope_table gives it; channels from ``rot`` on are not rotated.  Row t of
    request b is at position lens[b] + t, or with ``parents`` [B, T-1] (as the tree calls take it) lens[b] + its depth.
    ``interleaved``: channels 2i and 2i + 1 are a pair, otherwise i and i + rot / 2.  ``n_rows`` [B]: live rows of each
    request, the others give zeros.  ``out`` = dict(q=..., k=..., row_status=...); q and k there may be the inputs themselves.
    Returns that dict.
    """
    lib = load()
    at = _at(q)
    if k.get_device() != at:
        _not_at(k, at)
    dtype, like_q, like_k, table = q.dtype, q.shape, k.shape, rope.shape
    if len(like_q) != 4 or len(like_k) != 4 or k.dtype is not dtype:
        raise ValueError("q and k must be [B, T, heads, head_dim] of one dtype")
    B, T, hq, dim = like_q
    B1, T1, hkv, dim1 = like_k
    if B1 != B or T1 != T or dim1 != dim:
        raise ValueError("q and k must be [B, T, heads, head_dim] of one dtype")
    dt = wdt = _round_dtype(dtype, "q", (SPEC_BF16, SPEC_F16))
    if len(table) != 2:
        raise ValueError("rope must be [positions, rot]")
    if q_weight is not None or k_weight is not None:
        if q_weight is None or k_weight is None:
            raise ValueError("q_weight and k_weight come together")
        weights = q_weight.dtype
        wdt = _round_dtype(weights, "q_weight", (SPEC_F32, dt))
        wq, wk = _arg(q_weight, weights, (dim,), "the weights", at), _arg(k_weight, weights, (dim,), "the weights", at)
    else:
        wq = wk = None
    ln = _arg(lens, _I32, (B,), "lens", at)
    if out is None:
        y, z, status = _like(q, stream), _like(k, stream), _like(lens, stream)
        out = {"q": y, "k": z, "row_status": status}
        ys = zs = None
        status = status.data_ptr()
    else:
        y, z = out["q"], out["k"]
        for x, like in ((y, like_q), (z, like_k)):
            if x.shape != like or x.dtype is not dtype:
                raise ValueError("out['q'] and out['k'] must have the inputs' shapes and dtype")
            if x.get_device() != at:
                _not_at(x, at)
        ys, zs, status = _strides(y, 3), _strides(z, 3), _arg(out.get("row_status"), _I32, (B,), "row_status", at)
    rc = lib.qk_norm_rope(
        q.data_ptr(), _strides(q, 3), k.data_ptr(), _strides(k, 3), dt, B, T, hq, hkv, dim, wq, wk, wdt, eps,
        _arg(rope, _F32, table, "rope", at), table[0], table[1], interleaved, ln,
        _arg(parents, _I32, (B, T - 1), "parents", at) if T > 1 else None, _arg(n_rows, _I32, (B,), "n_rows", at),
        y.data_ptr(), ys, z.data_ptr(), zs, status, _raw_stream(stream, at))
    if rc:
        _check(rc)
    return out


def _pages_args(page_table, held, lens, free_pages, free_count, at):
    if page_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("page_table must be [B, width], free_pages [capacity]")
    B, width = page_table.shape
    cap = free_pages.shape[0]
    return (B, width, cap, _arg(page_table, _I32, (B, width), "page_table", at), _arg(held, _I32, (B,), "held", at),
            _arg(lens, _I32, (B,), "lens", at), _arg(free_pages, _I32, (cap,), "free_pages", at),
            _arg(free_count, _I32, (1,), "free_count", at))


def kv_pages_reserve(page_table, held, lens, free_pages, free_count, *, page_size: int, max_new: int, n_new=None, out=None,
                     stream=None):
    """Pages for the requests' next rows, from a free list on the GPU, and the rows' slots.

    ``free_pages`` [capacity] and ``free_count`` [1]: the free list, a stack; ``held`` [B]: the pages each request holds in
    page_table [B, width]; all int32, and page_table, held and free_count are written in place.  Request b gets the pages
    that its lens[b] + n_new[b] tokens need beside those held (``n_new`` [B] int32, at most ``max_new``, which holds without
    it), in the requests' order.  Returns dict(slots [B, max_new] int64: page * page_size + offset of each new row, -1 where there is none;
    row_status: ROW_NO_PAGES where the list was too short, and the request's pages are as before).
    """
    lib = load()
    at = _at(page_table)
    B, width, cap, table, hold, ln, free, count = _pages_args(page_table, held, lens, free_pages, free_count, at)
    _int(max_new, "max_new")
    if out is None:
        out = {"slots": _new((B, max_new), torch.int64, page_table.device, stream), "row_status": _like(held, stream)}
    rc = lib.kv_pages_reserve(
        table, width, hold, ln, _arg(n_new, _I32, (B,), "n_new", at), B, max_new, _int(page_size, "page_size"), free, cap, count,
        _arg(out.get("slots"), torch.int64, (B, max_new), "slots", at), _arg(out.get("row_status"), _I32, (B,), "row_status", at),
        _raw_stream(stream, at))
    if rc:
        _check(rc)
    return out


def kv_pages_release(page_table, held, lens, free_pages, free_count, *, page_size: int, out=None, stream=None):
    """Gives the pages past the requests' lengths back to the free list: those of a round's rejected rows, or with
    lens[b] = 0 all of an ended request's.  ``held``, ``free_pages`` and ``free_count`` are written in place (see
    kv_pages_reserve).  Returns dict(row_status)."""
    lib = load()
    at = _at(page_table)
    B, width, cap, table, hold, ln, free, count = _pages_args(page_table, held, lens, free_pages, free_count, at)
    if out is None:
        out = {"row_status": _like(held, stream)}
    rc = lib.kv_pages_release(table, width, hold, ln, B, _int(page_size, "page_size"), free, cap, count,
                              _arg(out.get("row_status"), _I32, (B,), "row_status", at), _raw_stream(stream, at))
    if rc:
        _check(rc)
    return out


def sample_logits(logits, uniforms, *, temperature=None, top_k=None, top_p=None, min_p=None, logprob: bool = True, out=None,
                  stream=None):
    """Draws one token a row, as the verify calls process the same logits.

    logits [N, V] (bf16 or fp32; any row stride, so one row expanded to N will do), ``uniforms`` [N] fp32 in [0, 1).  Settings per row, each [N] or None
    (off): ``temperature`` fp32 (0: the largest logit's token, otherwise 1e-30 to 1e30), ``top_k`` int32 (0: off; ties are kept), ``top_p`` fp32
    (>= 1: off; whole groups of equal logits, inclusive), ``min_p`` fp32 (0: off), applied in this order.  Mask tokens with -inf: a large
    finite number is right too, but slower with ``top_k`` in fp32.  Returns dict(tokens [N] int32, row_status and, with ``logprob``,
    logprob [N]: the ln of the token's probability among the kept ones).
    """
    lib = load()
    at = _at(logits)
    if logits.dim() != 2:
        raise ValueError("logits must be [N, V]")
    N, V = logits.shape
    dt = _round_dtype(logits.dtype, "logits", (SPEC_F32, SPEC_BF16))
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("the last dimension must be contiguous")
    stride = logits.stride(0) if N > 1 else V
    one = (N,)
    noise = _arg(uniforms, _F32, one, "uniforms", at)
    if out is None:
        tokens = _new(N, _I32, logits.device, stream)
        out = {"tokens": tokens, "row_status": _like(tokens, stream)}
        if logprob:
            out["logprob"] = _like(uniforms, stream)
    tokens = _arg(out["tokens"], _I32, one, "tokens", at)
    rc = lib.sample_logits(
        logits.data_ptr(), stride, dt, N, V, noise,
        _arg(temperature, _F32, one, "temperature", at), _arg(top_k, _I32, one, "top_k", at), _arg(top_p, _F32, one, "top_p", at),
        _arg(min_p, _F32, one, "min_p", at), tokens, _arg(out.get("logprob"), _F32, one, "logprob", at),
        _arg(out.get("row_status"), _I32, one, "row_status", at), _raw_stream(stream, at))
    if rc:
        _check(rc)
    return out
