"""The operators that complete a served decode step (C: include/qmm_serve.h).

qmm_kv4_append, qmm_kv4_read and qmm_attn_kv4 (a 4-bit paged cache), qmm_moe
(a mixture-of-experts layer) and qmm_sample, in the same manner as attn.py:
tensors supply pointers, strides and sizes, and the library checks and runs. All
tensors of a call are on one GPU, which need not be the current one; work is
enqueued on `stream`, or on that GPU's current stream.
"""
from __future__ import annotations

import ctypes
import threading

import block_quantized_matmul_amd as _qmm
from . import attn as _attn
from .attn import _PAIRS, _Place, _floats, _heads, _host_doubles, _ints, _ptr, _type

QMM_KV4_MAX_PAGE_TOKENS = 256
QMM_MOE_MAX_TOKENS = 16
QMM_MOE_MAX_EXPERTS = 512
QMM_MOE_MAX_USED = 32
QMM_SAMPLE_MAX_VOCAB = 524287

__all__ = ["QMM_KV4_MAX_PAGE_TOKENS", "QMM_MOE_MAX_TOKENS", "QMM_MOE_MAX_EXPERTS", "QMM_MOE_MAX_USED",
           "QMM_SAMPLE_MAX_VOCAB", "qmm_kv4_page_bytes", "qmm_kv4_append", "qmm_kv4_read", "qmm_attn_kv4",
           "qmm_attn_kv4_workspace_bytes", "qmm_attn_kv4_workspace_max_bytes", "qmm_moe", "qmm_moe_workspace_bytes",
           "qmm_sample", "qmm_sample_workspace_bytes"]

_vp, _i32, _i64, _f32, _f64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double
_ready = None
_loading = threading.Lock()
torch = None  # imported with the library, at the first call

_SIGNATURES = {  # restype, then the arguments; host structs travel as bytes
    "qmm_kv4_page_bytes": (_i64, [_i64] * 3),
    "qmm_kv4_append": (_i32, [_i32, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _f64, _vp, _vp, _i64, _i32, _vp, _vp, _i64,
                              _i64, _vp]),
    "qmm_kv4_read": (_i32, [_i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp]),
    "qmm_attn_kv4": (_i32, [_i32, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _f32, _vp,
                            _i64, _vp]),
    "qmm_attn_kv4_workspace_bytes": (_i64, [_i64] * 6),
    "qmm_moe": (_i32, [_vp, _i32, _i64, _i64, _vp, _i64, _i64, _i32, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _i64,
                       _i64, _vp, _vp, _vp, _vp, _i64, _vp]),
    "qmm_moe_workspace_bytes": (_i64, [_i64] * 5),
    "qmm_sample": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp]),
    "qmm_sample_workspace_bytes": (_i64, [_i64] * 2),
}


def _lib():
    return _ready or _load()


def _load():
    """Declares the functions, once, whichever thread comes first: what others find is complete."""
    global _ready, torch
    with _loading:
        if _ready is None:
            _attn._lib()
            import torch
            L = _qmm.lib()
            for name, (res, args) in _SIGNATURES.items():
                f = getattr(L, name)
                f.argtypes, f.restype = args, res
            _ready = L
    return _ready


def _pages(cache, page_tokens, n_kv_heads, head_dim):
    """The number of pages of a cache: a contiguous uint8 tensor [n_pages][qmm_kv4_page_bytes(...)]."""
    if cache.dtype is not torch.uint8 or cache.dim() != 2 or not cache.is_contiguous():
        raise TypeError("cache must be a contiguous 2-D uint8 tensor")
    size = _ready.qmm_kv4_page_bytes(page_tokens, n_kv_heads, head_dim)
    if size < 0:
        raise _qmm.QmmError(int(size), "qmm_kv4_page_bytes")
    if cache.shape[1] != size:
        raise ValueError(f"a page of the cache holds {cache.shape[1]} bytes, the call needs {size}")
    return cache.shape[0]


def qmm_kv4_page_bytes(page_tokens: int, n_kv_heads: int, head_dim: int) -> int:
    """Bytes of a page of a 4-bit cache with room for page_tokens tokens (16, 32, 64, 128 or 256)."""
    size = int(_lib().qmm_kv4_page_bytes(int(page_tokens), int(n_kv_heads), int(head_dim)))
    if size < 0:
        raise _qmm.QmmError(size, "qmm_kv4_page_bytes")
    return size


def qmm_kv4_append(K, V, cache, page_tokens, slots, positions=None, freqs=None, pairs="halves", norm=False, weight=None,
                   eps=1e-6, stream=None):
    """Keys (normed, rotated) and values into a 4-bit paged cache (C: qmm_kv4_append).

    K and V [n_tokens][n_kv_heads][head_dim], fp32, fp16 or bf16, any strides with
    contiguous heads; cache uint8 [n_pages][qmm_kv4_page_bytes(...)]; slots int32
    [n_tokens]: page * page_tokens + place, or outside the cache for a token that
    is not stored. positions int32 [n_tokens] and freqs (the host table of radians
    per position, as for qmm_norm_rope) rotate the keys, norm and weight (fp32
    [head_dim]) norm them first. Returns the cache."""
    L = _lib()
    place = _Place(stream, ("K", "V", "cache", "slots", "positions", "weight"), (K, V, cache, slots, positions, weight))
    if K.dim() != 3:
        raise ValueError("K and V must be [n_tokens][n_kv_heads][head_dim]")
    shape, dtype = K.shape, K.dtype
    n, heads, dim = shape
    n_pages = _pages(cache, page_tokens, heads, dim)
    if pairs not in _PAIRS:
        raise ValueError("pairs must be 'halves' or 'neighbours'")
    if weight is not None:
        if not norm:
            raise ValueError("weight needs norm")
        _floats(weight, "weight", (dim,))
    if (positions is None) != (freqs is None):
        raise ValueError("pass positions and freqs together")
    if positions is not None:
        _ints(positions, "positions", n)
    _ints(slots, "slots", n)
    fp, n_freqs, _keep = _host_doubles(freqs)
    place.run(L.qmm_kv4_append, "qmm_kv4_append", _type(K, "K"), _heads(K, "K", shape, dtype),
              _heads(V, "V", shape, dtype), n, heads, dim, bool(norm), _ptr(weight), eps, _ptr(positions), fp, n_freqs,
              _PAIRS[pairs], slots.data_ptr(), cache.data_ptr(), n_pages, page_tokens)
    return cache


def qmm_kv4_read(cache, page_tokens, slots, n_kv_heads=None, head_dim=None, dtype=None, K=None, V=None, stream=None):
    """The keys and values at slots of a 4-bit paged cache (C: qmm_kv4_read).

    Outputs [n][n_kv_heads][head_dim] fp32, fp16 or bf16: those that are passed,
    or both, new, of n_kv_heads, head_dim and dtype (float32). A slot outside the
    cache reads as NaNs. Returns (K, V), None for one that was not asked for."""
    L = _lib()
    place = _Place(stream, ("cache", "slots", "K", "V"), (cache, slots, K, V))
    _ints(slots, "slots", None)
    n = slots.shape[0]
    if K is None and V is None:
        if n_kv_heads is None or head_dim is None:
            raise ValueError("pass K, V or both, or n_kv_heads and head_dim")
        dtype = dtype or torch.float32
        K, V = (place.empty((n, n_kv_heads, head_dim), dtype) for _ in range(2))
    like = K if K is not None else V
    if like.dim() != 3:
        raise ValueError("K and V must be [n][n_kv_heads][head_dim]")
    _, heads, dim = like.shape
    n_pages = _pages(cache, page_tokens, heads, dim)
    shape = (n, heads, dim)
    place.run(L.qmm_kv4_read, "qmm_kv4_read", _type(like, "K"),
              None if K is None else _heads(K, "K", shape, like.dtype),
              None if V is None else _heads(V, "V", shape, like.dtype), n, heads, dim, slots.data_ptr(),
              cache.data_ptr(), n_pages, page_tokens)
    return K, V


def qmm_attn_kv4_workspace_bytes(n_rows: int, n_q_heads: int, n_kv_heads: int, head_dim: int, table_width: int,
                                 page_tokens: int) -> int:
    return int(_lib().qmm_attn_kv4_workspace_bytes(int(n_rows), int(n_q_heads), int(n_kv_heads), int(head_dim),
                                                   int(table_width), int(page_tokens)))


def qmm_attn_kv4_workspace_max_bytes(head_dim: int) -> int:
    """What no qmm_attn_kv4 call with heads of head_dim (64 or 128) needs more than."""
    if head_dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128")
    return 2048 * (1024 // head_dim) * (head_dim + 4) * 4 + 16 * 1024


def qmm_attn_kv4(Q, cache, page_tokens, n_kv_heads, tables, lengths, scale=None, O=None, workspace=None, stream=None):
    """Attention of a decode batch over a 4-bit paged cache (C: qmm_attn_kv4).

    Q [n_rows][n_q_heads][head_dim], fp16 or bf16, any strides (multiples of 8
    elements) with contiguous heads; cache as qmm_kv4_append fills it; tables int32
    [n_rows][table_width], the pages of each row's sequence in order (rows of any
    stride, so an expanded table serves several tokens of one sequence); lengths
    int32 [n_rows], the tokens each row attends to. A length outside the table, or
    a page outside the cache, gives that row NaNs; a length of 0 zeros. scale
    defaults to head_dim ** -0.5. O (like Q) is allocated if None. Without a
    workspace, one of qmm_attn_kv4_workspace_bytes bytes is allocated."""
    L = _lib()
    place = _Place(stream, ("Q", "cache", "tables", "lengths", "O", "workspace"),
                   (Q, cache, tables, lengths, O, workspace))
    if Q.dim() != 3:
        raise ValueError("Q must be [n_rows][n_q_heads][head_dim]")
    shape, dtype = Q.shape, Q.dtype
    n, hq, dim = shape
    n_pages = _pages(cache, page_tokens, n_kv_heads, dim)
    if tables.dtype is not torch.int32 or tables.dim() != 2 or (tables.shape[1] > 1 and tables.stride(1) != 1):
        raise TypeError("tables must be a 2-D int32 tensor with contiguous rows")
    if tables.shape[0] != n:
        raise ValueError(f"tables holds {tables.shape[0]} rows, the call needs {n}")
    _ints(lengths, "lengths", n)
    if O is None:
        O = place.empty(shape, dtype)
    width = tables.shape[1]
    _keep, ws, ws_bytes = place.workspace(workspace,
                                          L.qmm_attn_kv4_workspace_bytes(n, hq, n_kv_heads, dim, width, page_tokens),
                                          "qmm_attn_kv4_workspace_bytes")
    place.run(L.qmm_attn_kv4, "qmm_attn_kv4", _type(Q, "Q"), _heads(Q, "Q", shape, dtype), _heads(O, "O", shape, dtype), n,
              hq, n_kv_heads, dim, cache.data_ptr(), n_pages, page_tokens, tables.data_ptr(), tables.stride(0), width,
              lengths.data_ptr(), dim ** -0.5 if scale is None else scale, ws, ws_bytes)
    return O


def qmm_moe_workspace_bytes(n_tokens: int, k: int, n_ff: int, n_experts: int, n_used: int) -> int:
    return int(_lib().qmm_moe_workspace_bytes(int(n_tokens), int(k), int(n_ff), int(n_experts), int(n_used)))


def _stack(W, name, n_experts, n_rows):
    """(row stride, expert stride) of a uint8 tensor [n_experts][n_rows][bytes] with contiguous rows."""
    if W.dtype is not torch.uint8 or W.dim() != 3:
        raise TypeError(f"{name} must be a uint8 tensor [n_experts][n_rows][row bytes]")
    if W.shape[0] != n_experts or W.shape[1] != n_rows:
        raise ValueError(f"{name} must hold {n_experts} experts of {n_rows} rows, got {list(W.shape)}")
    if W.shape[2] > 1 and W.stride(2) != 1:
        raise ValueError(f"the bytes of one row of {name} must be contiguous")
    nb1 = W.stride(1) if n_rows > 1 else max(W.stride(1), W.shape[2])
    nb2 = W.stride(0) if n_experts > 1 else max(W.stride(0), n_rows * nb1)
    return nb1, nb2


def _row_fits(W, name, qtype, k):
    """The rows hold k weights of the type, and the two bytes behind an odd number of 2-byte-aligned blocks."""
    need = _qmm.qmm_row_bytes(qtype, k)
    if need >= 0 and W.shape[2] < (need + 3) // 4 * 4:
        raise ValueError(f"a row of {name} holds {W.shape[2]} bytes, {k} weights need {(need + 3) // 4 * 4}")


def qmm_moe(X, router, gate, up, type_in, down, type_out, n_used, renormalise=True, Y=None, ids=None, weights=None,
            workspace=None, stream=None):
    """A mixture-of-experts layer of up to QMM_MOE_MAX_TOKENS tokens (C: qmm_moe):
    Y[t] = sum over the n_used experts of largest logits router X[t] of
    w down_e (silu(gate_e X[t]) * (up_e X[t])).

    X fp32 or fp16 [n_tokens][k], router fp32 [n_experts][k], both contiguous;
    gate and up uint8 [n_experts][n_ff][row bytes], blocks of type_in, with one
    pair of strides; down uint8 [n_experts][k][row bytes], blocks of type_out;
    their rows and experts at any strides that are multiples of 4 bytes. ids
    (int32) and weights (fp32) [n_tokens][n_used], if given, receive the choice.
    Y (fp32 [n_tokens][k]) is allocated if None; without a workspace, one of
    qmm_moe_workspace_bytes bytes is allocated. Returns Y."""
    L = _lib()
    place = _Place(stream, ("X", "router", "gate", "up", "down", "Y", "ids", "weights", "workspace"),
                   (X, router, gate, up, down, Y, ids, weights, workspace))
    if X.dtype is not torch.float32 and X.dtype is not torch.float16:
        raise TypeError("X must be float32 or float16")
    if X.dim() != 2 or not X.is_contiguous() or router.dim() != 2:
        raise ValueError("X must be contiguous [n_tokens][k], router [n_experts][k]")
    (n, k), experts = X.shape, router.shape[0]
    _floats(router, "router", (experts, k))
    if gate.dim() != 3:
        raise TypeError("gate must be a uint8 tensor [n_experts][n_ff][row bytes]")
    ff = gate.shape[1]
    strides = _stack(gate, "gate", experts, ff)
    if _stack(up, "up", experts, ff) != strides:
        raise ValueError("gate and up must have the same strides")
    out_strides = _stack(down, "down", experts, k)
    for W, name, qtype, width in ((gate, "gate", type_in, k), (up, "up", type_in, k), (down, "down", type_out, ff)):
        _row_fits(W, name, qtype, width)
    if Y is None:
        Y = place.empty((n, k), torch.float32)
    else:
        _floats(Y, "Y", (n, k))
    if ids is not None and (ids.dtype is not torch.int32 or ids.shape != (n, n_used) or not ids.is_contiguous()):
        raise TypeError("ids must be a contiguous int32 tensor [n_tokens][n_used]")
    if weights is not None:
        _floats(weights, "weights", (n, n_used))
    _keep, ws, ws_bytes = place.workspace(workspace, L.qmm_moe_workspace_bytes(n, k, ff, experts, n_used),
                                          "qmm_moe_workspace_bytes")
    place.run(L.qmm_moe, "qmm_moe", X.data_ptr(), _attn.QMM_T_F32 if X.dtype is torch.float32 else _attn.QMM_T_F16, n, k,
              router.data_ptr(), experts, n_used, bool(renormalise), gate.data_ptr(), up.data_ptr(), type_in, ff, *strides,
              down.data_ptr(), type_out, *out_strides, Y.data_ptr(), _ptr(ids), _ptr(weights), ws, ws_bytes)
    return Y


def qmm_sample_workspace_bytes(n_rows: int, vocab: int) -> int:
    return int(_lib().qmm_sample_workspace_bytes(int(n_rows), int(vocab)))


def qmm_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, probs=None, workspace=None,
               stream=None):
    """The next token of every row of logits (C: qmm_sample).

    logits [n_rows][vocab] fp32, fp16 or bf16, contiguous rows at any stride; u fp32
    [n_rows], random numbers from [0, 1); temperature, top_p and min_p fp32 [n_rows],
    top_k int32 [n_rows], each None for none. Of the tokens in the order of falling
    logits, the first top_k, of those the shortest beginning that holds top_p of
    their probability, and of those the ones above min_p of the largest are kept, and
    the one where the sum of probabilities passes u is taken. tokens (int32
    [n_rows]) is allocated if None; -1 where no logit is above -infinity. probs (fp32
    [n_rows]), if given, receives the probabilities among what was kept. Without a
    workspace, one of qmm_sample_workspace_bytes bytes is allocated. Returns tokens."""
    L = _lib()
    place = _Place(stream, ("logits", "u", "temperature", "top_k", "top_p", "min_p", "tokens", "probs", "workspace"),
                   (logits, u, temperature, top_k, top_p, min_p, tokens, probs, workspace))
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [n_rows][vocab] with contiguous rows")
    n, vocab = logits.shape
    for t, name in ((u, "u"), (temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p"), (probs, "probs")):
        if t is not None:
            _floats(t, name, (n,))
    if top_k is not None:
        _ints(top_k, "top_k", n)
    if tokens is None:
        tokens = place.empty((n,), torch.int32)
    else:
        _ints(tokens, "tokens", n)
    _keep, ws, ws_bytes = place.workspace(workspace, L.qmm_sample_workspace_bytes(n, vocab), "qmm_sample_workspace_bytes")
    place.run(L.qmm_sample, "qmm_sample", logits.data_ptr(), _type(logits, "logits"), n, vocab, logits.stride(0),
              u.data_ptr(), _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p), tokens.data_ptr(), _ptr(probs),
              ws, ws_bytes)
    return tokens
