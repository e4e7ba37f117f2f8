"""The operators between the MUL_MATs of a served layer (C: include/qmm_attn.h).

qmm_lora, qmm_norm_rope, qmm_attn_prompt and qmm_attn_shared, as a ctypes
binding that only marshals arguments, like the package's other functions:
tensors supply pointers, strides and sizes, and the library checks and runs.
All tensors of a call are on one GPU, which need not be the current one; work
is enqueued on `stream`, or on that GPU's current stream. Memory a call
allocates (an output or a workspace that was not passed) belongs to the call's
stream, and an output may also be used on the current one (after waiting for
the call).
"""
from __future__ import annotations

import ctypes
import struct
import threading
from typing import NamedTuple, Optional

import block_quantized_matmul_amd as _qmm

QMM_T_F32 = 0
QMM_T_F16 = 1
QMM_T_BF16 = 2
QMM_ROPE_HALVES = 0
QMM_ROPE_NEIGHBOURS = 1
QMM_LORA_MAX_RANK = 256
QMM_HEAD_PARTS_MAX = 4
QMM_NORM_ROPE_MAX_DIM = 512

__all__ = ["QMM_T_F32", "QMM_T_F16", "QMM_T_BF16", "QMM_ROPE_HALVES", "QMM_ROPE_NEIGHBOURS", "QMM_LORA_MAX_RANK",
           "QMM_HEAD_PARTS_MAX", "QMM_NORM_ROPE_MAX_DIM", "qmm_head_part", "qmm_heads_desc", "qmm_head_part_desc",
           "qmm_lora", "qmm_lora_workspace_bytes", "qmm_lora_workspace_max_bytes", "qmm_norm_rope", "qmm_attn_prompt",
           "qmm_attn_shared", "qmm_attn_shared_workspace_bytes", "qmm_attn_shared_workspace_max_bytes"]

_PART_NAMES = ("X", "Y", "weight") + ("positions", "slots") + ("X", "Y", "weight") * (QMM_HEAD_PARTS_MAX - 1)
_PAIRS = {"halves": QMM_ROPE_HALVES, "neighbours": QMM_ROPE_NEIGHBOURS}
_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class qmm_heads_desc(ctypes.Structure):
    """Mirror of the C struct qmm_heads (include/qmm_attn.h)."""
    _fields_ = [("data", _vp), ("seq_stride", _i64), ("token_stride", _i64), ("head_stride", _i64)]


class qmm_head_part_desc(ctypes.Structure):
    """Mirror of the C struct qmm_head_part (include/qmm_attn.h)."""
    _fields_ = [("X", _vp), ("x_type", _i32), ("x_token_stride", _i64), ("x_head_stride", _i64), ("Y", _vp),
                ("y_type", _i32), ("y_row_stride", _i64), ("y_head_stride", _i64), ("n_heads", _i64), ("norm", _i32),
                ("weight", _vp), ("rotate", _i32), ("slotted", _i32)]


class qmm_head_part(NamedTuple):
    """One group of heads of a qmm_norm_rope call: X [n_tokens][n_heads][head_dim]
    to Y [n_tokens or n_slots][n_heads][head_dim], any strides with contiguous
    heads, each fp32, fp16 or bf16; weight fp32 [head_dim]."""
    X: object
    Y: object
    norm: bool = False
    weight: Optional[object] = None
    rotate: bool = False
    slotted: bool = False


_ready = None
_loading = threading.Lock()
_types = {}
_calls = {}
torch = None  # imported with the library, at the first call
_part_bytes = struct.Struct("@PiqqPiqqqiPii0P").pack  # a qmm_head_part_desc's
_heads_bytes = struct.Struct("@Pqqq").pack  # a qmm_heads_desc's


def _lib():
    return _ready or _load()


def _load():
    """Declares the functions, once, whichever thread comes first: what others find is complete."""
    global _ready, torch
    with _loading:
        if _ready is None:
            import torch
            _types.update({torch.float32: QMM_T_F32, torch.float16: QMM_T_F16, torch.bfloat16: QMM_T_BF16})
            L = _qmm.lib()
            heads = ctypes.POINTER(qmm_heads_desc)
            L.qmm_lora.argtypes = [_vp, _i32, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
            L.qmm_lora.restype = _i32
            L.qmm_lora_workspace_bytes.argtypes = [_i64, _i64, _i64]
            L.qmm_lora_workspace_bytes.restype = _i64
            L.qmm_norm_rope.argtypes = [ctypes.POINTER(qmm_head_part_desc), _i32, _i64, _i64, _f32, _vp, _vp, _i64, _i32,
                                        _vp, _i64, _vp]
            L.qmm_norm_rope.restype = _i32
            L.qmm_attn_prompt.argtypes = [_i32, heads, heads, heads, heads, _i64, _i64, _i64, _i64, _vp, _i64, _f32, _vp]
            L.qmm_attn_prompt.restype = _i32
            L.qmm_attn_shared.argtypes = [_i32, heads, heads, heads, _i64, heads, heads, _i64, _vp, heads, _i64, _i64,
                                          _i64, _i64, _f32, _vp, _i64, _vp]
            L.qmm_attn_shared.restype = _i32
            L.qmm_attn_shared_workspace_bytes.argtypes = [_i64] * 6
            L.qmm_attn_shared_workspace_bytes.restype = _i64
            # the same functions for this module, which passes host structs as bytes
            for name in ("qmm_norm_rope", "qmm_attn_prompt", "qmm_attn_shared"):
                f = L[name]
                f.argtypes = [_vp if issubclass(t, ctypes._Pointer) else t for t in getattr(L, name).argtypes]
                f.restype = _i32
                _calls[name] = f
            _ready = L
    return _ready


def _refuse(named):
    """Raises what is wrong with the places of a call's (name, tensor) pairs."""
    first = None
    for name, t in named:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a GPU tensor (the library has no CPU path)")
        if first is None:
            first = t.device
        elif t.device != first:
            raise ValueError(f"{name} is on {t.device}, other tensors of the call on {first}")
    raise TypeError("a call needs GPU tensors")


class _Place:
    """Where a call runs: the one GPU of its tensors and the stream's handle.
    (These calls are short, so this takes the cheapest route to each answer.)"""
    __slots__ = ("device", "handle", "foreign", "like")

    def __init__(self, stream, names, tensors):
        try:
            device = tensors[0].get_device()
            for t in tensors:
                if t is not None and t.get_device() != device:
                    _refuse(zip(names, tensors))
        except AttributeError:
            device = -1
        if device < 0:
            _refuse(zip(names, tensors))
        self.device, self.like = device, tensors[0]
        self.handle = torch._C._cuda_getCurrentRawStream(device)
        self.foreign = None
        if stream is not None:
            if stream.device.index != device:  # (whose handle may be the same: default streams')
                raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
            if stream.cuda_stream != self.handle:
                self.handle, self.foreign = stream.cuda_stream, stream

    def empty(self, shape, dtype):
        if self.foreign is None:
            return self.like.new_empty(shape, dtype=dtype)
        # memory of the call's stream: what the current one freed may still be written by work enqueued there
        with torch.cuda.stream(self.foreign):
            t = self.like.new_empty(shape, dtype=dtype)
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def workspace(self, given, need, what):
        """The call's workspace (the caller's, or a new one), its pointer and size."""
        if need < 0:
            raise _qmm.QmmError(int(need), what)
        if given is None:
            if need == 0:
                return None, None, 0
            given = self.empty(need, torch.uint8)
        elif given.dtype != torch.uint8 or not given.is_contiguous():
            raise TypeError("workspace must be a contiguous uint8 tensor")
        return given, given.data_ptr(), given.numel()

    def run(self, function, what, *args):
        """The library's function with the tensors' GPU current."""
        if torch._C._cuda_getDevice() == self.device:
            status = function(*args, self.handle)
        else:
            with torch.cuda.device(self.device):
                status = function(*args, self.handle)
        if status != 0:
            raise _qmm.QmmError(status, what)


def _type(t, name):
    code = _types.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has an unsupported type {t.dtype}")
    return code


def _ints(t, name, n):
    """A contiguous int32 vector of n elements (None: any number)."""
    shape = t.shape
    if t.dtype is not torch.int32 or len(shape) != 1 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous 1-D int32 tensor")
    if n is not None and shape[0] != n:
        raise ValueError(f"{name} holds {shape[0]} elements, the call needs {n}")


def _floats(t, name, shape):
    if t.dtype is not torch.float32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _strides(t, name):
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1 and t.numel() > 0:
        raise ValueError(f"the elements of one head of {name} must be contiguous")
    return st


def _heads(t, name, shape, dtype):
    """qmm_heads (as bytes) of a tensor of `shape`: [tokens][heads][dim] or [seqs][tokens][heads][dim]."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    st = _strides(t, name)
    return _heads_bytes(t.data_ptr(), st[0] if len(st) == 4 else 0, st[-3], st[-2])


def _ptr(t):
    return None if t is None else t.data_ptr()


def qmm_lora_workspace_bytes(n_tokens: int, k: int, rank: int) -> int:
    return int(_lib().qmm_lora_workspace_bytes(int(n_tokens), int(k), int(rank)))


def qmm_lora_workspace_max_bytes(max_tokens: int, max_k: int, max_rank: int) -> int:
    """What no qmm_lora call of at most these sizes needs more than: for a workspace kept for calls of different sizes
    (qmm_lora_workspace_bytes may be larger for fewer tokens). The header's inline function."""
    rows = min(max_tokens, 512) * min(max(max_k // 512, 16), 256)
    if max_tokens > 512:
        rows = max(rows, 32768)
    return max(rows, max_tokens) * max_rank * 4


def qmm_lora(X, A, B, ids, scales=None, base=None, Y=None, workspace=None, stream=None):
    """Low-rank adapters of many requests beside a shared projection (C: qmm_lora):
    Y[t] = base[t] + scales[a] * B[a] (A[a] X[t]) with a = ids[t].

    X fp32 or fp16 [n_tokens][k]; A fp16 [n_adapters][rank][k], B fp16
    [n_adapters][n_rows][rank], ids int32 [n_tokens] (-1: no adapter, any other
    id outside the stack: a row of NaNs), scales fp32 [n_adapters] or None for
    1, base fp32 [n_tokens][n_rows] or None for zeros; all contiguous. Y (fp32
    [n_tokens][n_rows]) is allocated if None, and may be base. Without a
    workspace, one of qmm_lora_workspace_bytes bytes is allocated."""
    L = _lib()
    place = _Place(stream, ("X", "A", "B", "ids", "scales", "base", "Y", "workspace"),
                   (X, A, B, ids, scales, base, Y, workspace))
    if X.dtype is not torch.float32 and X.dtype is not torch.float16:
        raise TypeError("X must be float32 or float16")
    if X.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("X must be [n_tokens][k], A [n_adapters][rank][k], B [n_adapters][n_rows][rank]")
    (n, k), (n_adapters, rank, ka), (nb, n_rows, rank_b) = X.shape, A.shape, B.shape
    if ka != k or nb != n_adapters or rank_b != rank:
        raise ValueError("X must be [n_tokens][k], A [n_adapters][rank][k], B [n_adapters][n_rows][rank]")
    if A.dtype is not torch.float16 or B.dtype is not torch.float16:
        raise TypeError("A and B must be float16")
    if not (X.is_contiguous() and A.is_contiguous() and B.is_contiguous()):
        raise ValueError("X, A and B must be contiguous")
    _ints(ids, "ids", n)
    if scales is not None:
        _floats(scales, "scales", (n_adapters,))
    if base is not None:
        _floats(base, "base", (n, n_rows))
    if Y is None:
        Y = place.empty((n, n_rows), torch.float32)
    else:
        _floats(Y, "Y", (n, n_rows))
    _keep, ws, ws_bytes = place.workspace(workspace, L.qmm_lora_workspace_bytes(n, k, rank),
                                          "qmm_lora_workspace_bytes")
    place.run(L.qmm_lora, "qmm_lora", X.data_ptr(), QMM_T_F32 if X.dtype is torch.float32 else QMM_T_F16, n, k,
              A.data_ptr(), B.data_ptr(), n_adapters, rank, n_rows, _ptr(scales), ids.data_ptr(), _ptr(base),
              Y.data_ptr(), ws, ws_bytes)
    return Y


def _host_doubles(freqs):
    """(pointer, count, object that owns the memory) of the host table of frequencies."""
    if freqs is None:
        return None, 0, None
    if isinstance(freqs, torch.Tensor):
        if freqs.is_cuda or freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
            raise TypeError("freqs must be a contiguous 1-D float64 host tensor or a sequence of numbers")
        return freqs.data_ptr(), freqs.shape[0], freqs
    own = (ctypes.c_double * len(freqs))(*(float(f) for f in freqs))
    return ctypes.addressof(own), len(freqs), own


def qmm_norm_rope(parts, positions=None, freqs=None, pairs="halves", eps=1e-6, slots=None, stream=None):
    """Norm, rotation, conversion and store of a batch's heads (C: qmm_norm_rope).

    parts: up to QMM_HEAD_PARTS_MAX qmm_head_part, all of one n_tokens and
    head_dim; every Y is preallocated. positions int32 [n_tokens] on the GPU;
    freqs the host table of radians per position (a float64 tensor or a
    sequence), read during the call; pairs "halves" or "neighbours"; slots
    int32 [n_tokens], the rows of the slotted parts' Y (one outside it: the
    token is not stored). Returns the Ys."""
    _lib()
    parts = [p if isinstance(p, qmm_head_part) else qmm_head_part(*p) for p in parts]
    if not parts:
        return []
    if len(parts) > QMM_HEAD_PARTS_MAX:
        raise ValueError(f"at most {QMM_HEAD_PARTS_MAX} parts")
    if pairs not in _PAIRS:
        raise ValueError("pairs must be 'halves' or 'neighbours'")
    place = _Place(stream, _PART_NAMES, [parts[0].X, parts[0].Y, parts[0].weight, positions, slots]
                   + [t for p in parts[1:] for t in (p.X, p.Y, p.weight)])
    if parts[0].X.dim() != 3:
        raise ValueError("X must be [n_tokens][n_heads][head_dim]")
    n, _, dim = parts[0].X.shape
    vector = (dim,)
    descs = b""
    n_slots = None
    for X, Y, norm, weight, rotate, slotted in parts:
        xs, ys = X.shape, Y.shape
        if len(xs) != 3 or xs[0] != n or xs[2] != dim:
            raise ValueError("every X must be [n_tokens][n_heads][head_dim] with one n_tokens and head_dim")
        if len(ys) != 3 or ys[1] != xs[1] or ys[2] != dim or (not slotted and ys[0] != n):
            raise ValueError("Y must be [n_tokens][n_heads][head_dim], or [n_slots][...] if slotted")
        if slotted:
            if slots is None:
                raise ValueError("a slotted part needs slots")
            if n_slots is not None and ys[0] != n_slots:
                raise ValueError("slotted parts must have one number of slots")
            n_slots = ys[0]
        if rotate and (positions is None or freqs is None):
            raise ValueError("a rotated part needs positions and freqs")
        if weight is not None:
            if not norm:
                raise ValueError("weight needs norm")
            _floats(weight, "weight", vector)
        xst, yst = X.stride(), Y.stride()
        if xst[2] != 1 or yst[2] != 1:
            _strides(X, "X"), _strides(Y, "Y")
        xt, yt = _types.get(X.dtype), _types.get(Y.dtype)
        if xt is None or yt is None:
            _type(X, "X"), _type(Y, "Y")
        descs += _part_bytes(X.data_ptr(), xt, xst[0], xst[1], Y.data_ptr(), yt, yst[0], yst[1], xs[1], bool(norm),
                             0 if weight is None else weight.data_ptr(), bool(rotate), bool(slotted))
    if positions is not None:
        _ints(positions, "positions", n)
    if slots is not None:
        _ints(slots, "slots", n)
    fp, n_freqs, _keep = _host_doubles(freqs)
    place.run(_calls["qmm_norm_rope"], "qmm_norm_rope", descs, len(parts), n, dim, eps, _ptr(positions), fp, n_freqs,
              _PAIRS[pairs], _ptr(slots), n_slots or 0)
    return [p.Y for p in parts]


def qmm_attn_prompt(Q, K, V, seq_starts, scale=None, O=None, stream=None):
    """Causal attention over packed prompts (C: qmm_attn_prompt).

    Q [n_tokens][n_q_heads][head_dim], K and V [n_tokens][n_kv_heads][head_dim],
    fp16 or bf16, any strides (multiples of 8 elements) with contiguous heads;
    seq_starts int32 [n_seqs + 1] on the GPU: sequence i holds tokens
    seq_starts[i] .. seq_starts[i + 1] - 1. scale defaults to
    head_dim ** -0.5. O (like Q) is allocated if None; rows of tokens outside
    every sequence are not written."""
    _lib()
    place = _Place(stream, ("Q", "K", "V", "seq_starts", "O"), (Q, K, V, seq_starts, O))
    if Q.dim() != 3 or K.dim() != 3:
        raise ValueError("Q must be [n_tokens][n_q_heads][head_dim], K and V [n_tokens][n_kv_heads][head_dim]")
    shape, dtype = Q.shape, Q.dtype
    n, hq, dim = shape
    hkv = K.shape[1]
    _ints(seq_starts, "seq_starts", None)
    if seq_starts.shape[0] < 1:
        raise ValueError("seq_starts must hold n_seqs + 1 elements")
    if O is None:
        O = place.empty(shape, dtype)
    kv = (n, hkv, dim)
    place.run(_calls["qmm_attn_prompt"], "qmm_attn_prompt", _type(Q, "Q"), _heads(Q, "Q", shape, dtype),
              _heads(K, "K", kv, dtype), _heads(V, "V", kv, dtype), _heads(O, "O", shape, dtype), n, hq, hkv, dim,
              seq_starts.data_ptr(), seq_starts.shape[0] - 1, dim ** -0.5 if scale is None else scale)
    return O


def qmm_attn_shared_workspace_bytes(n_seqs: int, prefix_len: int, own_cap: int, n_q_heads: int, n_kv_heads: int,
                                    head_dim: int) -> int:
    return int(_lib().qmm_attn_shared_workspace_bytes(int(n_seqs), int(prefix_len), int(own_cap), int(n_q_heads),
                                                      int(n_kv_heads), int(head_dim)))


def qmm_attn_shared_workspace_max_bytes(max_seqs: int, n_q_heads: int, head_dim: int) -> int:
    """What no qmm_attn_shared call of at most max_seqs sequences needs more than, whatever the prefix and the caches: for
    a workspace kept for calls of different sizes (qmm_attn_shared_workspace_bytes may be larger for fewer sequences or
    keys). The header's inline function."""
    return (512 * (128 + 32) + 3 * max_seqs * n_q_heads) * (head_dim + 2) * 4


def qmm_attn_shared(Q, PK, PV, K, V, lengths, scale=None, O=None, workspace=None, stream=None):
    """Attention of a decode batch over a shared prefix, then each sequence's own
    cache (C: qmm_attn_shared).

    Q [n_seqs][n_q_heads][head_dim], one token of each sequence; PK and PV
    [prefix_len][n_kv_heads][head_dim], or None for no prefix; K and V
    [n_seqs][own_cap][n_kv_heads][head_dim] with lengths int32 [n_seqs], or all
    three None for no own caches; fp16 or bf16, any strides (multiples of 8
    elements) with contiguous heads. A length outside [0, own_cap] gives rows
    of NaNs. scale defaults to head_dim ** -0.5. O (like Q) is allocated if
    None. Without a workspace, one of qmm_attn_shared_workspace_bytes bytes is
    allocated."""
    L = _lib()
    place = _Place(stream, ("Q", "PK", "PV", "K", "V", "lengths", "O", "workspace"),
                   (Q, PK, PV, K, V, lengths, O, workspace))
    if (PK is None) != (PV is None) or (K is None) != (V is None) or (K is None) != (lengths is None):
        raise ValueError("pass PK and PV together, and K, V and lengths together")
    if Q.dim() != 3 or (PK is not None and PK.dim() != 3) or (K is not None and K.dim() != 4):
        raise ValueError("Q must be [n_seqs][n_q_heads][head_dim], PK and PV [prefix_len][n_kv_heads][head_dim], "
                         "K and V [n_seqs][own_cap][n_kv_heads][head_dim]")
    if PK is None and K is None:
        raise ValueError("pass a prefix, own caches or both")
    shape, dtype = Q.shape, Q.dtype
    n, hq, dim = shape
    prefix, cap = (0 if PK is None else PK.shape[0]), (0 if K is None else K.shape[1])
    hkv = PK.shape[1] if PK is not None else K.shape[2]
    if O is None:
        O = place.empty(shape, dtype)
    pk = pv = k = v = None
    if PK is not None:
        pk, pv = _heads(PK, "PK", (prefix, hkv, dim), dtype), _heads(PV, "PV", (prefix, hkv, dim), dtype)
    if K is not None:
        own = (n, cap, hkv, dim)
        k, v = _heads(K, "K", own, dtype), _heads(V, "V", own, dtype)
        _ints(lengths, "lengths", n)
    _keep, ws, ws_bytes = place.workspace(workspace, L.qmm_attn_shared_workspace_bytes(n, prefix, cap, hq, hkv, dim),
                                          "qmm_attn_shared_workspace_bytes")
    place.run(_calls["qmm_attn_shared"], "qmm_attn_shared", _type(Q, "Q"), _heads(Q, "Q", shape, dtype), pk, pv,
              prefix, k, v, cap, _ptr(lengths), _heads(O, "O", shape, dtype), n, hq, hkv, dim,
              dim ** -0.5 if scale is None else scale, ws, ws_bytes)
    return O
