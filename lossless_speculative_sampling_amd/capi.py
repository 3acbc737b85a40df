"""Thin ctypes binding of libspecverify.so (include/specverify.h), same names as the C ABI.

Argument marshalling only: torch tensors supply device pointers and the current HIP stream;
every step of the path runs in the library's kernels.  There is no CPU fallback - a missing
or unloadable library raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libspecverify.so")

SPEC_OK, SPEC_EINVAL, SPEC_EDTYPE, SPEC_EWORKSPACE, SPEC_EHIP = 0, -1, -2, -3, -4
SPEC_FP32, SPEC_BF16, SPEC_FP16, SPEC_E4M3, SPEC_FP64 = 0, 1, 2, 3, 4
SPEC_SAMPLE_DRAFT = 1
SPEC_UNIFORM_DRAFT = 2
SPEC_ASSISTED = 4
SPEC_POINT_DRAFT = 8
SPEC_ROPE_INTERLEAVED = 1
SPEC_MAX_F = 64
SPEC_MAX_KAPPA = 16
SPEC_NOALLOC_SCRATCH_BYTES = 32 << 20
ST_EMPTY_RESIDUAL = 8
ST_OUTSIDE_DRAFT_SUPPORT = 16
ST_BAD_LOGIT = 32
ST_BAD_TOKEN = 64
ST_DEGENERATE_DOWNWEIGHT = 128
ST_BAD_PARAM = 256
ST_PLACEMENT = 512
ST_BAD_PROB = 1024
ST_BAD_SLOT = 2048

EXPORTS = ("spec_workspace_bytes", "spec_verify", "saguaro_downweight", "saguaro_fanout", "saguaro_cache_build",
           "saguaro_cache_lookup", "saguaro_verify_cache", "saguaro_backup_plan", "mirror_signpost_workspace_bytes",
           "mirror_signposts", "mirror_tree_lookup", "pyramid_verify", "spec_read_ceiling",
           "saguaro_verify_cache_noalloc", "saguaro_verify_cache_lookup", "saguaro_verify_cache_lookup_timed",
           "spec_verify_probs_workspace_bytes", "spec_verify_probs", "spec_tree_rows", "spec_rope_frequencies",
           "spec_kv_append", "spec_prefix_attention_workspace_bytes", "spec_prefix_attention")

_P = ctypes.c_void_p
_I = ctypes.c_int
_U64 = ctypes.c_uint64
_I64 = ctypes.c_int64
_D = ctypes.c_double
_F = ctypes.c_float


class _Cache(ctypes.Structure):
    """spec_kv_cache of the C ABI."""
    _fields_ = [("k", _P), ("v", _P), ("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_stride", _I64), ("token_stride", _I64), ("head_stride", _I64), ("k_scale", _P), ("v_scale", _P)]


class SpecError(RuntimeError):
    def __init__(self, fn: str, rc: int):
        names = {SPEC_EINVAL: "SPEC_EINVAL", SPEC_EDTYPE: "SPEC_EDTYPE", SPEC_EWORKSPACE: "SPEC_EWORKSPACE",
                 SPEC_EHIP: "SPEC_EHIP"}
        super().__init__(f"{fn} returned {names.get(rc, rc)}")
        self.rc = rc


class Lib:
    def __init__(self, path: str = LIB_PATH):
        if not os.path.exists(path):
            raise RuntimeError(f"HIP library {path} is not built (python -m lossless_speculative_sampling_amd.build)")
        self.cdll = L = ctypes.CDLL(path)
        L.spec_workspace_bytes.argtypes = [_I, _I, _I]
        L.spec_workspace_bytes.restype = ctypes.c_size_t
        L.spec_verify.argtypes = [_P, _I, _P, _I, _I, _I, _I, _P, _I, ctypes.c_float, _P, _U64, _U64, ctypes.c_uint32,
                                  _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.saguaro_downweight.argtypes = [_P, _I, _I, _I, _I, _I, _P, _I, ctypes.c_float, _P, _P, _P, _P, _P]
        L.saguaro_fanout.argtypes = [_I, _I, _D, _D, _P]
        L.saguaro_cache_build.argtypes = [_P, _I, _I, _I, _I, _P, _I, _D, _D, _P, _P, _P]
        L.saguaro_cache_lookup.argtypes = [_I, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P]
        L.saguaro_backup_plan.argtypes = [_I, _P, _P, _I, _P, _P, _P]
        L.mirror_signpost_workspace_bytes.argtypes = [_I, _I, _I]
        L.mirror_signpost_workspace_bytes.restype = ctypes.c_size_t
        L.mirror_signposts.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.mirror_tree_lookup.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]
        L.pyramid_verify.argtypes = [_P, _I, _P, _I, _I, _I, _I, _P, _I, ctypes.c_float, _P, _P, ctypes.c_uint64,
                                     ctypes.c_uint64, ctypes.c_uint32, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.saguaro_verify_cache.argtypes = [_P, _P, _I, _I, _I, _I, _P, _I, ctypes.c_float, _P, _U64, _U64,
                                           ctypes.c_uint32, _I, _D, _D, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t,
                                           _P]
        L.spec_read_ceiling.argtypes = [_P, ctypes.c_size_t, _P, _P]
        L.saguaro_verify_cache_lookup.argtypes = [_P, _P, _I, _I, _I, _I, _P, _I, ctypes.c_float, _P, _U64, _U64,
                                                  ctypes.c_uint32, _I, _D, _D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                                  ctypes.c_size_t, _P]
        L.saguaro_verify_cache_lookup_timed.argtypes = L.saguaro_verify_cache_lookup.argtypes + [_P, _P]
        L.saguaro_verify_cache_noalloc.argtypes = [_P, _P, _I, _I, _I, _I, _P, _I, ctypes.c_float, _P, _U64, _U64,
                                                   ctypes.c_uint32, _I, _D, _D, _P, _P, _P, _P, _P, _P, _P]
        L.spec_verify_probs.argtypes = [_P, _I64, _I64, _P, _I64, _I64, _I, _I, _I, _I, _P, _P, _P, _P, _I,
                                        ctypes.c_uint32, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.spec_tree_rows.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P]
        L.spec_rope_frequencies.argtypes = [_I, _D, _D, _D, _D, _I, _P]
        L.spec_kv_append.argtypes = [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I, _I, _I, _I, _I,
                                     _P, _P, _P, _I, _F, ctypes.c_uint32, _P, _P, _P]
        L.spec_prefix_attention.argtypes = [_P, _I64, _I64, _I, _I, _I, _P, _I, _P, _P, _I, _P, _P, _I, _P, _F, _P,
                                            _I64, _I64, _P, _P, ctypes.c_size_t, _P]
        for fn in EXPORTS[1:]:
            getattr(L, fn).restype = _I
        L.spec_verify_probs_workspace_bytes.argtypes = [_I, _I]
        L.spec_prefix_attention_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I64, _I]
        for fn in ("spec_verify_probs_workspace_bytes", "spec_prefix_attention_workspace_bytes"):
            getattr(L, fn).restype = ctypes.c_size_t


_lib: Optional[Lib] = None


def load(path: str = LIB_PATH) -> Lib:
    global _lib
    if _lib is None:
        _lib = Lib(path)
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, rc: int):
    if rc != SPEC_OK:
        raise SpecError(fn, rc)


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SPEC_FP32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return SPEC_BF16
    raise ValueError(f"unsupported logit dtype {t.dtype}")


# ---- argument checks: every shape and dtype the C ABI assumes, so that a wrong tensor raises here
# instead of being read past its end by the library ----
def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _int32(name: str, t: Optional[torch.Tensor], shape: tuple):
    _need(t is not None, f"{name} is required")
    _need(t.dtype == torch.int32, f"{name} must be int32, got {t.dtype}")
    _need(tuple(t.shape) == tuple(shape), f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _params(params: torch.Tensor, B: int):
    _int32("params", params, (B, 3))


def _logits(name: str, t: torch.Tensor, dims: int = 3) -> int:
    _need(t.dim() == dims, f"{name} must be {dims}-D, got shape {tuple(t.shape)}")
    _need(all(n > 0 for n in t.shape), f"{name} has an empty dimension: {tuple(t.shape)}")
    return dtype_code(t)


def _verify_inputs(draft: Optional[torch.Tensor], target: torch.Tensor, K: int, params: torch.Tensor,
                   tokens: torch.Tensor, draft_rows=None) -> int:
    code = _logits("target", target)
    B, rows, V = target.shape
    _need(K >= 1 and rows == K + 1, f"target must hold K + 1 = {K + 1} rows per request, got {rows}")
    if draft is not None:
        _need(_logits("draft", draft) == code, "draft and target must have the same dtype")
        _need(draft.shape[0] == B and draft.shape[2] == V, f"draft {tuple(draft.shape)} does not match target "
                                                           f"{tuple(target.shape)}")
        allowed = (K, K + 1) if draft_rows is None else (draft_rows,)
        _need(draft.shape[1] in allowed, f"draft must hold {' or '.join(map(str, allowed))} rows, got {draft.shape[1]}")
    _params(params, B)
    _int32("tokens", tokens, (B, K))
    return code


def _verify_out(out, B: int):
    for name in ("k", "tstar", "status"):
        _int32(f"out.{name}", getattr(out, name), (B,))
    _need(out.resid_mass.dtype == torch.float32 and tuple(out.resid_mass.shape) == (B,), "out.resid_mass must be float32 [B]")


def _workspace(ws: torch.Tensor):
    _need(ws.dtype == torch.uint8 and ws.dim() == 1, "workspace must be a 1-D uint8 tensor")


def spec_workspace_bytes(B: int, K: int, V: int) -> int:
    return int(load().cdll.spec_workspace_bytes(B, K, V))


def params_tensor(temperature, top_k, top_p, device="cuda") -> torch.Tensor:
    """[B] spec_params packed as int32 words {float T, int32 top_k, float top_p}."""
    T = torch.as_tensor(temperature, dtype=torch.float32).reshape(-1)
    k = torch.as_tensor(top_k, dtype=torch.int32).reshape(-1)
    p = torch.as_tensor(top_p, dtype=torch.float32).reshape(-1)
    B = max(T.numel(), k.numel(), p.numel())
    T, k, p = T.expand(B), k.expand(B), p.expand(B)
    rec = torch.stack([T.view(torch.int32), k, p.view(torch.int32)], dim=1).contiguous()
    return rec.to(device)


def new_workspace(B: int, K: int, V: int, device="cuda") -> torch.Tensor:
    """Zero-filled spec_verify workspace (the library leaves it zero-filled after every call)."""
    return torch.zeros(max(spec_workspace_bytes(B, K, V), 1), dtype=torch.uint8, device=device)


@dataclass
class VerifyOut:
    k: torch.Tensor
    tstar: torch.Tensor
    resid_mass: torch.Tensor
    status: torch.Tensor
    tokens: torch.Tensor


def spec_verify(draft: Optional[torch.Tensor], target: torch.Tensor, K: int, params: torch.Tensor,
                tokens: torch.Tensor, F: int = 0, C: float = 1.0, seed: int = 0, round_: int = 0, flags: int = 0,
                workspace: Optional[torch.Tensor] = None, out: Optional[VerifyOut] = None, stream=None) -> VerifyOut:
    """draft [B][Kd][V] and target [B][K+1][V] device logits; tokens [B][K] int32 (in, or out under
    SPEC_SAMPLE_DRAFT).  With SPEC_UNIFORM_DRAFT draft may be None.  Returns the outputs (allocated
    here unless `out` is given)."""
    _need(draft is not None or bool(flags & SPEC_UNIFORM_DRAFT), "draft logits are required without SPEC_UNIFORM_DRAFT")
    code = _verify_inputs(draft, target, K, params, tokens)
    B, _, V = target.shape
    Kd = draft.shape[1] if draft is not None else K
    dev = target.device
    if out is None:
        out = VerifyOut(torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                        torch.empty(B, dtype=torch.float32, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                        tokens)
    _verify_out(out, B)
    if workspace is None:
        workspace = new_workspace(B, K, V, dev)
    _workspace(workspace)
    rc = load().cdll.spec_verify(_ptr(draft), Kd, _ptr(target), code, B, K, V, _ptr(params), F,
                                 ctypes.c_float(C), _ptr(tokens), seed, round_, flags, _ptr(out.k), _ptr(out.tstar),
                                 _ptr(out.resid_mass), _ptr(out.status), _ptr(workspace), workspace.numel(),
                                 _stream(stream))
    _check("spec_verify", rc)
    out.tokens = tokens
    return out


def saguaro_downweight(draft: torch.Tensor, K: int, params: torch.Tensor, F: int, C: float, want_probs=False,
                       stream=None):
    _logits("draft", draft)
    B, Kd, V = draft.shape
    _need(1 <= K <= Kd, f"K = {K} must lie in [1, {Kd}] (draft rows)")
    _params(params, B)
    dev = draft.device
    ids = torch.empty((B, K, max(F, 1)), dtype=torch.int32, device=dev)
    Z = torch.empty((B, K), dtype=torch.float32, device=dev)
    st = torch.empty((B, K), dtype=torch.int32, device=dev)
    probs = torch.empty((B, K, V), dtype=torch.float32, device=dev) if want_probs else None
    rc = load().cdll.saguaro_downweight(_ptr(draft), Kd, dtype_code(draft), B, K, V, _ptr(params), F,
                                        ctypes.c_float(C), _ptr(ids), _ptr(Z), _ptr(probs), _ptr(st), _stream(stream))
    _check("saguaro_downweight", rc)
    return ids[:, :, :F], Z, probs, st


def saguaro_fanout(K: int, budget: int, a: float, r: float) -> list[int]:
    buf = (ctypes.c_int32 * (K + 1))()
    _check("saguaro_fanout", load().cdll.saguaro_fanout(K, budget, a, r, ctypes.cast(buf, _P)))
    return list(buf)


def saguaro_cache_build(draft: torch.Tensor, K: int, tokens: torch.Tensor, budget: int, a: float, r: float,
                        stream=None):
    _logits("draft", draft)
    B, Kd, V = draft.shape
    _need(K >= 1 and Kd == K + 1, f"draft must hold K + 1 = {K + 1} rows per request, got {Kd}")
    _int32("tokens", tokens, (B, K))
    fan = (ctypes.c_int32 * (K + 1))()
    cache = torch.empty((B, max(budget, 1)), dtype=torch.int32, device=draft.device)
    rc = load().cdll.saguaro_cache_build(_ptr(draft), dtype_code(draft), B, K, V, _ptr(tokens), budget, a, r,
                                         ctypes.cast(fan, _P), _ptr(cache), _stream(stream))
    _check("saguaro_cache_build", rc)
    return cache[:, :budget], list(fan)


def saguaro_verify_cache(draft: torch.Tensor, target: torch.Tensor, K: int, params: torch.Tensor, tokens: torch.Tensor,
                         budget: int, a: float, r: float, F: int = 0, C: float = 1.0, seed: int = 0, round_: int = 0,
                         flags: int = 0, workspace: Optional[torch.Tensor] = None, out: Optional[VerifyOut] = None,
                         cache: Optional[torch.Tensor] = None, stream=None):
    """spec_verify + saguaro_cache_build in one pass; draft [B][K+1][V].  Returns (VerifyOut,
    cache [B][budget], fan-out list)."""
    code = _verify_inputs(draft, target, K, params, tokens, draft_rows=K + 1)
    B, Kd, V = draft.shape
    dev = draft.device
    if out is None:
        out = VerifyOut(torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                        torch.empty(B, dtype=torch.float32, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                        tokens)
    _verify_out(out, B)
    if workspace is None:
        workspace = new_workspace(B, K, V, dev)
    _workspace(workspace)
    if cache is None:
        cache = torch.empty((B, max(budget, 1)), dtype=torch.int32, device=dev)
    _need(cache.dtype == torch.int32 and cache.dim() == 2 and cache.shape[0] == B and cache.shape[1] >= budget,
          f"cache must be int32 [{B}][>= {budget}]")
    fan = (ctypes.c_int32 * (K + 1))()
    rc = load().cdll.saguaro_verify_cache(_ptr(draft), _ptr(target), code, B, K, V, _ptr(params), F,
                                          ctypes.c_float(C), _ptr(tokens), seed, round_, flags, budget, a, r,
                                          ctypes.cast(fan, _P), _ptr(out.k), _ptr(out.tstar), _ptr(out.resid_mass),
                                          _ptr(out.status), _ptr(cache), _ptr(workspace), workspace.numel(),
                                          _stream(stream))
    _check("saguaro_verify_cache", rc)
    out.tokens = tokens
    return out, cache[:, :budget], list(fan)


def saguaro_verify_cache_lookup(draft: torch.Tensor, target: torch.Tensor, K: int, params: torch.Tensor,
                                tokens: torch.Tensor, budget: int, a: float, r: float, F: int = 0, C: float = 1.0,
                                seed: int = 0, round_: int = 0, flags: int = 0, workspace: Optional[torch.Tensor] = None,
                                out: Optional[VerifyOut] = None, cache: Optional[torch.Tensor] = None, stream=None):
    """saguaro_verify_cache and the mode-0 lookup of its outcomes in one call.  Returns (VerifyOut,
    cache [B][budget], fan-out list, slot [B] int32, hit [B] uint8, batch [2] int32)."""
    code = _verify_inputs(draft, target, K, params, tokens, draft_rows=K + 1)
    B, Kd, V = draft.shape
    dev = draft.device
    if out is None:
        out = VerifyOut(torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                        torch.empty(B, dtype=torch.float32, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                        tokens)
    _verify_out(out, B)
    if workspace is None:
        workspace = new_workspace(B, K, V, dev)
    _workspace(workspace)
    if cache is None:
        cache = torch.empty((B, max(budget, 1)), dtype=torch.int32, device=dev)
    _need(cache.dtype == torch.int32 and cache.dim() == 2 and cache.shape[0] == B and cache.shape[1] >= budget,
          f"cache must be int32 [{B}][>= {budget}]")
    slot = torch.empty(B, dtype=torch.int32, device=dev)
    hit = torch.empty(B, dtype=torch.uint8, device=dev)
    batch = torch.empty(2, dtype=torch.int32, device=dev)
    fan = (ctypes.c_int32 * (K + 1))()
    rc = load().cdll.saguaro_verify_cache_lookup(_ptr(draft), _ptr(target), code, B, K, V, _ptr(params), F,
                                                 ctypes.c_float(C), _ptr(tokens), seed, round_, flags, budget, a, r,
                                                 ctypes.cast(fan, _P), _ptr(out.k), _ptr(out.tstar),
                                                 _ptr(out.resid_mass), _ptr(out.status), _ptr(cache), _ptr(slot),
                                                 _ptr(hit), _ptr(batch), _ptr(workspace), workspace.numel(),
                                                 _stream(stream))
    _check("saguaro_verify_cache_lookup", rc)
    out.tokens = tokens
    return out, cache[:, :budget], list(fan), slot, hit, batch


def saguaro_verify_cache_noalloc(draft: torch.Tensor, target: torch.Tensor, K: int, params: torch.Tensor,
                                 tokens: torch.Tensor, budget: int, a: float, r: float, out: VerifyOut,
                                 cache: torch.Tensor, F: int = 0, C: float = 1.0, seed: int = 0, round_: int = 0,
                                 flags: int = 0, stream=None):
    """saguaro_verify_cache on the library's static scratch (no workspace); the caller passes the
    outputs (out, cache [B][>= budget]).  Returns the fan-out list."""
    code = _verify_inputs(draft, target, K, params, tokens, draft_rows=K + 1)
    B, Kd, V = draft.shape
    _verify_out(out, B)
    _need(cache.dtype == torch.int32 and cache.dim() == 2 and cache.shape[0] == B and cache.shape[1] >= budget,
          f"cache must be int32 [{B}][>= {budget}]")
    fan = (ctypes.c_int32 * (K + 1))()
    rc = load().cdll.saguaro_verify_cache_noalloc(_ptr(draft), _ptr(target), code, B, K, V, _ptr(params), F,
                                                  ctypes.c_float(C), _ptr(tokens), seed, round_, flags, budget, a, r,
                                                  ctypes.cast(fan, _P), _ptr(out.k), _ptr(out.tstar),
                                                  _ptr(out.resid_mass), _ptr(out.status), _ptr(cache),
                                                  _stream(stream))
    _check("saguaro_verify_cache_noalloc", rc)
    return list(fan)


def saguaro_cache_lookup(mode: int, cache: torch.Tensor, fanout_or_shape, K: int, B: int, k: torch.Tensor,
                         tstar: torch.Tensor, stream=None):
    dev = cache.device
    fs_list = [int(x) for x in fanout_or_shape]
    _need(cache.dtype == torch.int32, "cache must be int32")
    if mode == 0:
        _need(len(fs_list) == K + 1, f"mode 0 takes K + 1 = {K + 1} fan-out entries, got {len(fs_list)}")
        _need(cache.dim() == 2 and cache.shape[0] == B, f"cache must be [{B}][budget]")
        _need(cache.shape[1] >= sum(fs_list), f"cache holds {cache.shape[1]} slots, the fan-out needs {sum(fs_list)}")
        per = 1
    elif mode == 1:
        _need(len(fs_list) == 2, "mode 1 takes {kappa, gamma}")
        _need(cache.numel() == B * fs_list[0] * fs_list[1], "branches must hold B * kappa * gamma tokens")
        per = fs_list[0]  # k and t* of every chain
    else:
        raise ValueError(f"unknown lookup mode {mode}")
    _need(k.numel() == B * per, f"k must hold {B * per} entries")
    _need(tstar.numel() == B * per, f"tstar must hold {B * per} entries")
    _need(k.dtype == torch.int32, "k must be int32")
    _need(tstar.dtype == torch.int32, "tstar must be int32")
    fs = (ctypes.c_int32 * len(fs_list))(*fs_list)
    slot = torch.empty(B, dtype=torch.int32, device=dev)
    hit = torch.empty(B, dtype=torch.uint8, device=dev)
    batch = torch.empty(2, dtype=torch.int32, device=dev)
    rc = load().cdll.saguaro_cache_lookup(mode, _ptr(cache), ctypes.cast(fs, _P), K, B, _ptr(k), _ptr(tstar),
                                          _ptr(slot), _ptr(hit), _ptr(batch), _stream(stream))
    _check("saguaro_cache_lookup", rc)
    return slot, hit, batch


def saguaro_backup_plan(hit: torch.Tensor, batch: torch.Tensor, b_star: int, stream=None):
    """(use_backup [B] int32, switch [1] int32) on the device: the batch-aware random-token fallback."""
    B = hit.shape[0]
    _need(hit.dtype == torch.uint8 and hit.dim() == 1, "hit must be uint8 [B]")
    _int32("batch", batch, (2,))
    use = torch.empty(B, dtype=torch.int32, device=hit.device)
    sw = torch.empty(1, dtype=torch.int32, device=hit.device)
    rc = load().cdll.saguaro_backup_plan(B, _ptr(hit), _ptr(batch), b_star, _ptr(use), _ptr(sw), _stream(stream))
    _check("saguaro_backup_plan", rc)
    return use, sw



def mirror_signpost_workspace_bytes(B: int, V: int, kappa: int) -> int:
    return int(load().cdll.mirror_signpost_workspace_bytes(B, V, kappa))


def new_signpost_workspace(B: int, V: int, kappa: int, device="cuda") -> torch.Tensor:
    n = mirror_signpost_workspace_bytes(B, V, kappa)
    if n == 0:
        raise SpecError("mirror_signpost_workspace_bytes", SPEC_EINVAL)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def mirror_signposts(logits: torch.Tensor, kappa: int, want_bf16: bool = False,
                     workspace: Optional[torch.Tensor] = None, out=None, stream=None):
    """Early-exit signposts of logits [B][V]: (ids [B][kappa] int32, log p~ [B][kappa] float32,
    log p~ as bf16 bits [B][kappa] int16 or None, status [B] int32)."""
    code = _logits("logits", logits, dims=2)
    B, V = logits.shape
    dev = logits.device
    if workspace is None:
        workspace = new_signpost_workspace(B, V, kappa, dev)
    _workspace(workspace)
    if out is None:
        out = (torch.empty((B, kappa), dtype=torch.int32, device=dev),
               torch.empty((B, kappa), dtype=torch.float32, device=dev),
               torch.empty((B, kappa), dtype=torch.int16, device=dev) if want_bf16 else None,
               torch.empty(B, dtype=torch.int32, device=dev))
    ids, lp, lp16, st = out
    rc = load().cdll.mirror_signposts(_ptr(logits), code, B, V, kappa, _ptr(ids), _ptr(lp), _ptr(lp16),
                                      _ptr(st), _ptr(workspace), workspace.numel(), _stream(stream))
    _check("mirror_signposts", rc)
    return out


def mirror_tree_lookup(tokens: torch.Tensor, parents: torch.Tensor, path: torch.Tensor, k: torch.Tensor,
                       tstar: torch.Tensor, stream=None):
    """Reuse node of the committed prefix in each request's draft tree [B][N]: (node [B], hit [B], batch [2])."""
    _need(tokens.dim() == 2, "tokens must be [B][N]")
    B, N = tokens.shape
    _int32("tokens", tokens, (B, N))
    _int32("parents", parents, (B, N))
    _need(path.dim() == 2 and path.shape[0] == B, "path must be [B][gamma]")
    gamma = path.shape[1]
    _int32("path", path, (B, gamma))
    _int32("k", k, (B,))
    _int32("tstar", tstar, (B,))
    dev = tokens.device
    node = torch.empty(B, dtype=torch.int32, device=dev)
    hit = torch.empty(B, dtype=torch.uint8, device=dev)
    batch = torch.empty(2, dtype=torch.int32, device=dev)
    rc = load().cdll.mirror_tree_lookup(_ptr(tokens), _ptr(parents), B, N, gamma, _ptr(path), _ptr(k), _ptr(tstar),
                                        _ptr(node), _ptr(hit), _ptr(batch), _stream(stream))
    _check("mirror_tree_lookup", rc)
    return node, hit, batch


def pyramid_verify(draft: Optional[torch.Tensor], verifier: torch.Tensor, K: int, params: torch.Tensor,
                   tau: torch.Tensor, tokens: torch.Tensor, F: int = 0, C: float = 1.0, seed: int = 0, round_: int = 0,
                   flags: int = 0, want_div: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """Fuzzy (PyramidSD) verification of one stage: (VerifyOut, divergences [B][K] or None)."""
    _need(draft is not None or bool(flags & SPEC_UNIFORM_DRAFT), "draft logits are required without SPEC_UNIFORM_DRAFT")
    code = _verify_inputs(draft, verifier, K, params, tokens)
    B, _, V = verifier.shape
    _need(tau.dtype == torch.float32 and tuple(tau.shape) == (B,), "tau must be float32 [B]")
    Kd = draft.shape[1] if draft is not None else K
    dev = verifier.device
    if workspace is None:
        workspace = new_workspace(B, K, V, dev)
    _workspace(workspace)
    out = VerifyOut(torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                    torch.empty(B, dtype=torch.float32, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                    tokens)
    div = torch.zeros((B, K), dtype=torch.float32, device=dev) if want_div else None
    rc = load().cdll.pyramid_verify(_ptr(draft), Kd, _ptr(verifier), code, B, K, V, _ptr(params), F,
                                    ctypes.c_float(C), _ptr(tau), _ptr(tokens), seed, round_, flags, _ptr(out.k),
                                    _ptr(out.tstar), _ptr(out.resid_mass), _ptr(out.status), _ptr(div),
                                    _ptr(workspace), workspace.numel(), _stream(stream))
    _check("pyramid_verify", rc)
    return out, div


# ---- the steps on either side of the verification.  These take strided tensors where the C ABI has
# strides, and run on the device of their tensors (its current stream unless `stream` is given),
# whichever device is current.  A call here is a few microseconds of GPU work at its smallest, so the
# checks are written to cost little: one comparison each, messages made only when one fails. ----
_HALF = {torch.bfloat16: SPEC_BF16, torch.float16: SPEC_FP16}
_PROBS = {torch.float32: SPEC_FP32, **_HALF}
_I32, _F32, _F64, _U8 = torch.int32, torch.float32, torch.float64, torch.uint8


def _on_one_device(dev: int, tensors):
    """Raises unless every given tensor lies on GPU `dev`."""
    if dev < 0:
        raise ValueError("device tensor expected")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("device tensor expected" if t.get_device() < 0 else
                             f"tensors lie on different devices: cuda:{dev} and cuda:{t.get_device()}")


def _whole(name: str, t: Optional[torch.Tensor], dtype: torch.dtype, shape: tuple):
    if t is None or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _need(t is not None, f"{name} is required")
        _need(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
        _need(tuple(t.shape) == shape, f"{name} must have shape {shape}, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")


def _strides(name: str, t: torch.Tensor) -> tuple:
    """The outer strides of a tensor whose last dimension is contiguous."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return st


def _call(fn: str, dev: int, stream, *args):
    """Calls the library with the stream last, on GPU `dev`."""
    here = torch._C._cuda_getDevice()
    if dev != here:
        with torch.cuda.device(dev):
            return _call(fn, dev, stream, *args)
    rc = getattr(load().cdll, fn)(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if rc != SPEC_OK:
        raise SpecError(fn, rc)


def _data(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _lend(stream, dev: int, *tensors):
    """Tensors allocated here for a stream that the caller named: their memory is not given away before
    that stream has passed the call."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


@dataclass
class ProbsOut:
    k: torch.Tensor           # [B] int32
    tstar: torch.Tensor       # [B] int32
    emitted: torch.Tensor     # [B][K+1] int32: accepted tokens, t*, then -1
    resid_mass: torch.Tensor  # [B] float32
    status: torch.Tensor      # [B] int32 status bits


@functools.lru_cache(maxsize=1024)
def spec_verify_probs_workspace_bytes(B: int, V: int) -> int:
    return int(load().cdll.spec_verify_probs_workspace_bytes(B, V))


def spec_verify_probs(draft: Optional[torch.Tensor], target: torch.Tensor, tokens: torch.Tensor, accept_u: torch.Tensor,
                      sample_v: torch.Tensor, draft_lens: Optional[torch.Tensor] = None, flags: int = 0,
                      workspace: Optional[torch.Tensor] = None, out: Optional[ProbsOut] = None, stream=None) -> ProbsOut:
    """Verification from given probabilities, draft [B][K][V] (None with SPEC_UNIFORM_DRAFT or
    SPEC_POINT_DRAFT) and target [B][K+1][V] in fp32, bf16 or fp16, and given random numbers accept_u
    [B][K] and sample_v [B] in fp32 or fp64; tokens [B][K] and draft_lens [B] int32."""
    code = _PROBS.get(target.dtype)
    if target.dim() != 3 or code is None:
        raise ValueError("target must be [B][K+1][V] in fp32, bf16 or fp16")
    B, rows, V = target.shape
    K = rows - 1
    if B < 1 or K < 1 or V < 1:
        raise ValueError(f"target {tuple(target.shape)} holds no drafted position")
    ts = _strides("target", target)
    ds = (0, 0)
    if draft is not None:
        if draft.dtype is not target.dtype or draft.shape != (B, K, V):
            _need(draft.dtype == target.dtype, "draft and target must have the same dtype")
            raise ValueError(f"draft must be {(B, K, V)}, got {tuple(draft.shape)}")
        ds = _strides("draft", draft)
    elif not flags:
        raise ValueError("draft probabilities are required without SPEC_UNIFORM_DRAFT or SPEC_POINT_DRAFT")
    _whole("tokens", tokens, _I32, (B, K))
    ut = accept_u.dtype
    if ut is not _F32 and ut is not _F64:
        raise ValueError("accept_u must be float32 or float64")
    _whole("accept_u", accept_u, ut, (B, K))
    _whole("sample_v", sample_v, ut, (B,))
    if draft_lens is not None:
        _whole("draft_lens", draft_lens, _I32, (B,))
    dev = target.get_device()
    if out is None:
        k, tstar, status, mass = torch.empty(4, B, dtype=_I32, device=target.device).unbind()
        out = ProbsOut(k, tstar, torch.empty(B, rows, dtype=_I32, device=target.device), mass.view(_F32), status)
    else:
        for name in ("k", "tstar", "status"):
            _whole(f"out.{name}", getattr(out, name), _I32, (B,))
        _whole("out.emitted", out.emitted, _I32, (B, rows))
        _whole("out.resid_mass", out.resid_mass, _F32, (B,))
    need = spec_verify_probs_workspace_bytes(B, V)
    if workspace is not None:
        _workspace(workspace)
    elif need:
        workspace = torch.empty(need, dtype=_U8, device=target.device)
    _on_one_device(dev, (target, draft, tokens, accept_u, sample_v, draft_lens, out.k, out.tstar, out.emitted,
                         out.resid_mass, out.status, workspace))
    if stream is not None:
        _lend(stream, dev, workspace, out.k, out.tstar, out.emitted, out.resid_mass, out.status)
    _call("spec_verify_probs", dev, stream, _data(draft), ds[0], ds[1], target.data_ptr(), ts[0], ts[1], code, B, K, V,
          tokens.data_ptr(), _data(draft_lens), accept_u.data_ptr(), sample_v.data_ptr(),
          SPEC_FP64 if ut is _F64 else SPEC_FP32, flags, out.k.data_ptr(), out.tstar.data_ptr(), out.emitted.data_ptr(),
          out.resid_mass.data_ptr(), out.status.data_ptr(), _data(workspace), 0 if workspace is None else workspace.numel())
    return out


@dataclass
class TreeRows:
    positions: torch.Tensor     # [B][N] int32, -1 outside the tree
    append_slots: torch.Tensor  # [B][N] int32, -1 outside the tree
    suffix_slots: torch.Tensor  # [B][N][max_depth] int32, root to node, then -1
    suffix_len: torch.Tensor    # [B][N] int32: the depth, 0 outside the tree


def spec_tree_rows(tokens: torch.Tensor, parents: torch.Tensor, slots: torch.Tensor, ctx_len: torch.Tensor,
                   max_depth: int, out: Optional[TreeRows] = None, stream=None) -> TreeRows:
    """The rows of draft trees [B][N] (parents first, as in mirror_tree_lookup) on contexts of ctx_len [B]
    tokens, node n of request b at cache slot slots[b][n]."""
    if tokens.dim() != 2:
        raise ValueError("tokens must be [B][N]")
    shape = B, N = tuple(tokens.shape)
    _whole("tokens", tokens, _I32, shape)
    _whole("parents", parents, _I32, shape)
    _whole("slots", slots, _I32, shape)
    _whole("ctx_len", ctx_len, _I32, (B,))
    if max_depth < 1:
        raise ValueError("max_depth must be at least 1")
    if out is None:
        pos, app, length = torch.empty(3, B, N, dtype=_I32, device=tokens.device).unbind()
        out = TreeRows(pos, app, torch.empty(B, N, max_depth, dtype=_I32, device=tokens.device), length)
    else:
        for name in ("positions", "append_slots", "suffix_len"):
            _whole(f"out.{name}", getattr(out, name), _I32, shape)
        _whole("out.suffix_slots", out.suffix_slots, _I32, (B, N, max_depth))
    dev = tokens.get_device()
    _on_one_device(dev, (tokens, parents, slots, ctx_len, out.positions, out.append_slots, out.suffix_slots, out.suffix_len))
    if stream is not None:
        _lend(stream, dev, out.positions, out.append_slots, out.suffix_slots, out.suffix_len)
    _call("spec_tree_rows", dev, stream, tokens.data_ptr(), parents.data_ptr(), slots.data_ptr(), ctx_len.data_ptr(), B, N,
          max_depth, out.positions.data_ptr(), out.append_slots.data_ptr(), out.suffix_slots.data_ptr(),
          out.suffix_len.data_ptr())
    return out


def spec_rope_frequencies(rot_dim: int, base: float = 10000.0, factor: float = 1.0, low: float = 1.0, high: float = 4.0,
                          original_len: int = 8192) -> list[float]:
    """Rotary inverse frequencies, those that turn slowly stretched by `factor` (1: none)."""
    buf = (ctypes.c_double * max(rot_dim // 2, 1))()
    _check("spec_rope_frequencies", load().cdll.spec_rope_frequencies(rot_dim, base, factor, low, high, original_len,
                                                                      ctypes.cast(buf, _P)))
    return list(buf)


@dataclass
class Rotary:
    freqs: torch.Tensor        # [rot_dim / 2] float64 on the device
    interleaved: bool = False  # pairs (2i, 2i + 1); otherwise (i, i + rot_dim / 2)
    scale: float = 1.0         # a factor on cos and sin


@dataclass
class KVCache:
    """A paged cache: k and v [num_pages][page_size][heads][head_dim], bf16, fp16 or float8_e4m3fn (with
    float32 scales [heads], None: 1); slot s is token s % page_size of page s // page_size.  Views with
    other strides will do, the same for k and v, as long as head_dim is contiguous."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None

    def described(self) -> _Cache:
        k, v, ks, vs = self.k, self.v, self.k_scale, self.v_scale
        shape, st = k.shape, k.stride()
        eight = k.dtype is torch.float8_e4m3fn
        code = SPEC_E4M3 if eight else _HALF.get(k.dtype)
        if len(shape) != 4 or v.shape != shape or v.dtype is not k.dtype or v.stride() != st or code is None:
            _need(k.dim() == 4 and k.shape == v.shape, "cache: k and v must be [num_pages][page_size][heads][head_dim] alike")
            _need(k.dtype == v.dtype, "cache: k and v must have the same dtype")
            _need(code is not None, f"cache: unsupported dtype {k.dtype}")
            raise ValueError("cache: k and v must have the same strides")
        if st[3] != 1 and shape[3] > 1:
            raise ValueError("cache: head_dim must be contiguous")
        if ks is not None or vs is not None:
            _need(eight, "cache: scales belong to an 8-bit cache")
            for name, x in (("k_scale", ks), ("v_scale", vs)):
                if x is not None:
                    _whole(f"cache.{name}", x, _F32, (shape[2],))
        return _Cache(k.data_ptr(), v.data_ptr(), code, *shape, *st[:3], _data(ks), _data(vs))


def spec_kv_append(k: Optional[torch.Tensor], v: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                   slots: Optional[torch.Tensor], cache: Optional[KVCache], rotary: Optional[Rotary] = None,
                   q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Rotates k [T][heads][head_dim] and stores it with v into the cache at slots [T] (int32, -1: none), and
    rotates q [T][q_heads][head_dim] into q_out (allocated here unless given; q itself: in place), which is
    returned.  k, v, slots and cache may all be None (queries only), and q (keys and values only)."""
    lead = q if q is not None else k
    if lead is None or lead.dim() != 3:
        raise ValueError("q or k must be given, as [T][heads][head_dim]")
    T, _, D = lead.shape
    code = _HALF.get(lead.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {lead.dtype}")
    desc, heads, q_heads, rot, rscale, rflags = None, 0, 0, 0, 1.0, 0
    freqs = ks = vs = qs = os = None
    if k is not None and v is not None and cache is not None and slots is not None:
        if k.dim() != 3 or v.shape != k.shape or k.dtype is not lead.dtype or v.dtype is not lead.dtype:
            _need(v.shape == k.shape, "k and v must have the same shape")
            _need(k.dim() == 3, "k must be [T][heads][head_dim]")
            raise ValueError("q, k and v must have the same dtype")
        heads = k.shape[1]
        if k.shape != (T, heads, D):
            raise ValueError(f"k must be [{T}][heads][{D}], got {tuple(k.shape)}")
        ks, vs = _strides("k", k), _strides("v", v)
        _whole("slots", slots, _I32, (T,))
        desc = cache.described()
        if desc.heads != heads or desc.head_dim != D:
            raise ValueError(f"cache heads {(desc.heads, desc.head_dim)} do not match k {(heads, D)}")
        of_cache = (cache.k, cache.v, cache.k_scale, cache.v_scale)
    else:
        _need(k is None and v is None and cache is None, "k, v, slots and cache come together")
        slots, of_cache, ks, vs = None, (), (0, 0), (0, 0)
    if q is not None:
        q_heads = q.shape[1]
        qs = _strides("q", q)
        if q_out is None:
            q_out = torch.empty(T, q_heads, D, dtype=q.dtype, device=q.device)
        elif q_out.shape != q.shape or q_out.dtype is not q.dtype:
            raise ValueError("q_out must be like q")
        os = _strides("q_out", q_out)
    else:
        q_out, qs, os = None, (0, 0), (0, 0)
    if rotary is not None:
        freqs = rotary.freqs
        rot = 2 * freqs.numel()
        _need(rot <= D, f"rotary.freqs must hold at most {D // 2} frequencies")
        _whole("rotary.freqs", freqs, _F64, (rot // 2,))
        _whole("positions", positions, _I32, (T,))
        rscale, rflags = rotary.scale, SPEC_ROPE_INTERLEAVED if rotary.interleaved else 0
    else:
        positions = None
    if status is not None:
        _whole("status", status, _I32, (T,))
    dev = lead.get_device()
    _on_one_device(dev, (lead, q_out, k, v, positions, slots, freqs, status, *of_cache))
    if stream is not None:
        _lend(stream, dev, q_out)
    _call("spec_kv_append", dev, stream, _data(q), qs[0], qs[1], _data(q_out), os[0], os[1], _data(k), ks[0], ks[1],
          _data(v), vs[0], vs[1], code, T, q_heads, heads, D, _data(positions), _data(slots), _data(freqs), rot, rscale,
          rflags, None if desc is None else ctypes.byref(desc), _data(status))
    return q_out


@functools.lru_cache(maxsize=1024)
def spec_prefix_attention_workspace_bytes(R: int, G: int, q_heads: int, heads: int, head_dim: int,
                                          max_prefix: int, max_suffix: int) -> int:
    return int(load().cdll.spec_prefix_attention_workspace_bytes(R, G, q_heads, heads, head_dim, max_prefix, max_suffix))


def spec_prefix_attention(q: torch.Tensor, cache: KVCache, page_table: Optional[torch.Tensor],
                          prefix_len: Optional[torch.Tensor], row_start: torch.Tensor,
                          suffix_slots: Optional[torch.Tensor] = None, suffix_len: Optional[torch.Tensor] = None,
                          scale: Optional[float] = None, out: Optional[torch.Tensor] = None, want_lse: bool = False,
                          lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of rows q [R][q_heads][head_dim] in groups row_start [G+1], each over its group's prefix
    (page_table [G][max_pages], prefix_len [G]) and its own suffix_slots [R][max_suffix], suffix_len [R].  scale:
    head_dim^-0.5 unless given.  Returns (out, lse); lse [R][q_heads] float32 with want_lse, else None.  Rows
    outside every group (padding) keep what out and lse held, so give both where there are such rows."""
    code = _HALF.get(q.dtype)
    if q.dim() != 3 or code is None:
        raise ValueError("q must be [R][q_heads][head_dim] in bf16 or fp16")
    R, Hq, D = q.shape
    qs = _strides("q", q)
    desc = cache.described()
    heads = desc.heads
    if desc.head_dim != D or heads < 1 or Hq % heads:
        raise ValueError(f"cache heads {(heads, desc.head_dim)} do not serve q {(Hq, D)}")
    G = row_start.numel() - 1
    if G < 1:
        raise ValueError("row_start must be [G+1]")
    _whole("row_start", row_start, _I32, (G + 1,))
    pages = S = 0
    if page_table is not None:
        if page_table.dim() != 2:
            raise ValueError("page_table must be [G][max_pages]")
        pages = page_table.shape[1]
        _whole("page_table", page_table, _I32, (G, pages))
        _whole("prefix_len", prefix_len, _I32, (G,))
    else:
        prefix_len = None
    if suffix_slots is not None:
        if suffix_slots.dim() != 2:
            raise ValueError("suffix_slots must be [R][max_suffix]")
        S = suffix_slots.shape[1]
        _whole("suffix_slots", suffix_slots, _I32, (R, S))
        _whole("suffix_len", suffix_len, _I32, (R,))
    else:
        suffix_len = None
    if out is None:
        out = torch.empty(R, Hq, D, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError("out must be like q")
    os = _strides("out", out)
    if lse is not None:
        _whole("lse", lse, _F32, (R, Hq))
    elif want_lse:
        lse = torch.empty(R, Hq, dtype=_F32, device=q.device)
    if workspace is None:
        workspace = torch.empty(spec_prefix_attention_workspace_bytes(R, G, Hq, heads, D, pages * desc.page_size, S),
                                dtype=_U8, device=q.device)
    else:
        _workspace(workspace)
    dev = q.get_device()
    _on_one_device(dev, (q, cache.k, cache.v, cache.k_scale, cache.v_scale, page_table, prefix_len, row_start,
                         suffix_slots, suffix_len, out, lse, workspace))
    if stream is not None:
        _lend(stream, dev, workspace, out, lse)
    _call("spec_prefix_attention", dev, stream, q.data_ptr(), qs[0], qs[1], code, R, Hq, ctypes.byref(desc), G,
          row_start.data_ptr(), _data(page_table), pages, _data(prefix_len), _data(suffix_slots), S, _data(suffix_len),
          D ** -0.5 if scale is None else scale, out.data_ptr(), os[0], os[1], _data(lse), workspace.data_ptr(),
          workspace.numel())
    return out, lse


def spec_read_ceiling(data: torch.Tensor, sink: torch.Tensor, stream: Optional[int] = None) -> None:
    """One plain streaming read of every byte of `data` (contiguous, 16-byte aligned, a multiple
    of 16 bytes): the bandwidth ceiling a call reading as many bytes is set against."""
    _need(data.is_contiguous(), "data must be contiguous")
    _need(sink.dtype == torch.int32 and sink.numel() >= 1, "sink must hold one int32")
    nbytes = data.numel() * data.element_size()
    rc = load().cdll.spec_read_ceiling(_ptr(data), nbytes, _ptr(sink), _stream(stream))
    _check("spec_read_ceiling", rc)
