"""The operators between the MUL_MATs of a served layer (C: include/qmm_attn.h).

qmm_lora, qmm_norm_rope, qmm_attn_prompt and qmm_attn_shared, as a ctypes
binding that only marshals arguments, like the package's other functions:
tensors supply pointers, strides and sizes, and the library checks and runs.
All tensors of a call are on one GPU, which need not be the current one; work
is enqueued on `stream`, or on that GPU's current stream. Memory a call
allocates (an output or a workspace that was not passed) is kept from reuse
until the stream has passed the call.
"""
from __future__ import annotations

import ctypes
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
           "qmm_lora", "qmm_lora_workspace_bytes", "qmm_norm_rope", "qmm_attn_prompt", "qmm_attn_shared",
           "qmm_attn_shared_workspace_bytes"]

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


def _lib():
    global _ready
    if _ready is None:
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
        _ready = L
    return _ready


class _Place:
    """Where a call runs: the one GPU of its tensors, made current for the
    duration of the call, and the stream."""
    __slots__ = ("device", "stream", "foreign", "guard")

    def __init__(self, stream, named):
        import torch
        device = None
        for name, t in named:
            if t is None:
                continue
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{name} must be a GPU tensor (the library has no CPU path)")
            if device is None:
                device = t.device
            elif t.device != device:
                raise ValueError(f"{name} is on {t.device}, other tensors of the call on {device}")
        current = torch.cuda.current_stream(device)
        if stream is None:
            stream = current
        elif stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        self.device, self.stream = device, stream
        self.foreign = stream.cuda_stream != current.cuda_stream
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def empty(self, shape, dtype):
        import torch
        t = torch.empty(shape, dtype=dtype, device=self.device)
        if self.foreign:
            t.record_stream(self.stream)
        return t

    def workspace(self, given, need, what):
        """Pointer and size of the call's workspace: the caller's, or a new one."""
        import torch
        if need < 0:
            raise _qmm.QmmError(int(need), what)
        if given is None:
            if need == 0:
                return None, 0, None
            given = self.empty((need,), torch.uint8)
        elif given.dtype != torch.uint8 or not given.is_contiguous():
            raise TypeError("workspace must be a contiguous uint8 tensor")
        return given.data_ptr(), given.numel(), given


def _type(t, name, allowed):
    import torch
    code = {torch.float32: QMM_T_F32, torch.float16: QMM_T_F16, torch.bfloat16: QMM_T_BF16}.get(t.dtype)
    if code is None or code not in allowed:
        raise TypeError(f"{name} has an unsupported type {t.dtype}")
    return code


def _ints(t, name, shape):
    """An int32 vector of a given length (None: any)."""
    import torch
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous 1-D int32 tensor")
    if shape is not None and t.shape[0] != shape:
        raise ValueError(f"{name} holds {t.shape[0]} elements, the call needs {shape}")


def _floats(t, name, shape):
    import torch
    if t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _stride(t, dim):
    # torch leaves the strides of one-element axes and empty tensors open; they are never used
    return t.stride(dim) if t.shape[dim] > 1 and t.numel() > 0 else 0


def _contiguous_heads(t, name):
    if t.shape[-1] > 1 and t.stride(-1) != 1 and t.numel() > 0:
        raise ValueError(f"the elements of one head of {name} must be contiguous")


def _heads(t, name, shape, dtype):
    """qmm_heads of a tensor of `shape`: [tokens][heads][dim] or [seqs][tokens][heads][dim]."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    _contiguous_heads(t, name)
    return qmm_heads_desc(t.data_ptr(), _stride(t, 0) if len(shape) == 4 else 0, _stride(t, -3), _stride(t, -2))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(status, what):
    if status != 0:
        raise _qmm.QmmError(status, what)


def qmm_lora_workspace_bytes(n_tokens: int, k: int, rank: int) -> int:
    return int(_lib().qmm_lora_workspace_bytes(int(n_tokens), int(k), int(rank)))


def qmm_lora(X, A, B, ids, scales=None, base=None, Y=None, workspace=None, stream=None):
    """Low-rank adapters of many requests beside a shared projection (C: qmm_lora):
    Y[t] = base[t] + scales[a] * B[a] (A[a] X[t]) with a = ids[t].

    X fp32 or fp16 [n_tokens][k]; A fp16 [n_adapters][rank][k], B fp16
    [n_adapters][n_rows][rank], ids int32 [n_tokens] (-1: no adapter, any other
    id outside the stack: a row of NaNs), scales fp32 [n_adapters] or None for
    1, base fp32 [n_tokens][n_rows] or None for zeros; all contiguous. Y (fp32
    [n_tokens][n_rows]) is allocated if None, and may be base. Without a
    workspace, one of qmm_lora_workspace_bytes bytes is allocated."""
    import torch
    with _Place(stream, (("X", X), ("A", A), ("B", B), ("ids", ids), ("scales", scales), ("base", base), ("Y", Y),
                         ("workspace", workspace))) as place:
        x_type = _type(X, "X", (QMM_T_F32, QMM_T_F16))
        if X.dim() != 2 or A.dim() != 3 or B.dim() != 3:
            raise ValueError("X must be [n_tokens][k], A [n_adapters][rank][k], B [n_adapters][n_rows][rank]")
        (n, k), (n_adapters, rank, ka), (nb, n_rows, rank_b) = X.shape, A.shape, B.shape
        if ka != k or nb != n_adapters or rank_b != rank:
            raise ValueError("X must be [n_tokens][k], A [n_adapters][rank][k], B [n_adapters][n_rows][rank]")
        if A.dtype != torch.float16 or B.dtype != torch.float16:
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
        L = _lib()
        ws, ws_bytes, _keep = place.workspace(workspace, L.qmm_lora_workspace_bytes(n, k, rank),
                                              "qmm_lora_workspace_bytes")
        _check(L.qmm_lora(X.data_ptr(), x_type, n, k, A.data_ptr(), B.data_ptr(), n_adapters, rank, n_rows,
                          _ptr(scales), ids.data_ptr(), _ptr(base), Y.data_ptr(), ws, ws_bytes,
                          place.stream.cuda_stream), "qmm_lora")
    return Y


def _host_doubles(freqs):
    """(pointer, count, object that owns the memory) of the host table of frequencies."""
    import torch
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
    parts = [p if isinstance(p, qmm_head_part) else qmm_head_part(*p) for p in parts]
    if not parts:
        return []
    if len(parts) > QMM_HEAD_PARTS_MAX:
        raise ValueError(f"at most {QMM_HEAD_PARTS_MAX} parts")
    if pairs not in _PAIRS:
        raise ValueError("pairs must be 'halves' or 'neighbours'")
    named = [("positions", positions), ("slots", slots)]
    for p in parts:
        named += [("X", p.X), ("Y", p.Y), ("weight", p.weight)]
    with _Place(stream, named) as place:
        if parts[0].X.dim() != 3:
            raise ValueError("X must be [n_tokens][n_heads][head_dim]")
        n, _, dim = parts[0].X.shape
        descs = (qmm_head_part_desc * len(parts))()
        n_slots = None
        every = (QMM_T_F32, QMM_T_F16, QMM_T_BF16)
        for d, p in zip(descs, parts):
            X, Y = p.X, p.Y
            if X.dim() != 3 or Y.dim() != 3 or X.shape[0] != n or X.shape[2] != dim:
                raise ValueError("every X must be [n_tokens][n_heads][head_dim] with one n_tokens and head_dim")
            if Y.shape[1] != X.shape[1] or Y.shape[2] != dim or (not p.slotted and Y.shape[0] != n):
                raise ValueError("Y must be [n_tokens][n_heads][head_dim], or [n_slots][...] if slotted")
            if p.slotted:
                if slots is None:
                    raise ValueError("a slotted part needs slots")
                if n_slots is not None and Y.shape[0] != n_slots:
                    raise ValueError("slotted parts must have one number of slots")
                n_slots = Y.shape[0]
            if p.rotate and (positions is None or freqs is None):
                raise ValueError("a rotated part needs positions and freqs")
            if p.weight is not None:
                if not p.norm:
                    raise ValueError("weight needs norm")
                _floats(p.weight, "weight", (dim,))
            _contiguous_heads(X, "X")
            _contiguous_heads(Y, "Y")
            d.X, d.x_type, d.x_token_stride, d.x_head_stride = X.data_ptr(), _type(X, "X", every), _stride(X, 0), _stride(X, 1)
            d.Y, d.y_type, d.y_row_stride, d.y_head_stride = Y.data_ptr(), _type(Y, "Y", every), _stride(Y, 0), _stride(Y, 1)
            d.n_heads, d.norm, d.weight, d.rotate, d.slotted = X.shape[1], p.norm, _ptr(p.weight), p.rotate, p.slotted
        if positions is not None:
            _ints(positions, "positions", n)
        if slots is not None:
            _ints(slots, "slots", n)
        fp, n_freqs, _keep = _host_doubles(freqs)
        _check(_lib().qmm_norm_rope(descs, len(parts), n, dim, eps, _ptr(positions), fp, n_freqs, _PAIRS[pairs],
                                    _ptr(slots), n_slots or 0, place.stream.cuda_stream), "qmm_norm_rope")
    return [p.Y for p in parts]


def qmm_attn_prompt(Q, K, V, seq_starts, scale=None, O=None, stream=None):
    """Causal attention over packed prompts (C: qmm_attn_prompt).

    Q [n_tokens][n_q_heads][head_dim], K and V [n_tokens][n_kv_heads][head_dim],
    fp16 or bf16, any strides (multiples of 8 elements) with contiguous heads;
    seq_starts int32 [n_seqs + 1] on the GPU: sequence i holds tokens
    seq_starts[i] .. seq_starts[i + 1] - 1. scale defaults to
    head_dim ** -0.5. O (like Q) is allocated if None; rows of tokens outside
    every sequence are not written."""
    with _Place(stream, (("Q", Q), ("K", K), ("V", V), ("seq_starts", seq_starts), ("O", O))) as place:
        if Q.dim() != 3 or K.dim() != 3:
            raise ValueError("Q must be [n_tokens][n_q_heads][head_dim], K and V [n_tokens][n_kv_heads][head_dim]")
        n, hq, dim = Q.shape
        hkv = K.shape[1]
        t = _type(Q, "Q", (QMM_T_F16, QMM_T_BF16))
        _ints(seq_starts, "seq_starts", None)
        if seq_starts.shape[0] < 1:
            raise ValueError("seq_starts must hold n_seqs + 1 elements")
        if O is None:
            O = place.empty((n, hq, dim), Q.dtype)
        q, k, v, o = (_heads(x, name, (n, h, dim), Q.dtype)
                      for x, name, h in ((Q, "Q", hq), (K, "K", hkv), (V, "V", hkv), (O, "O", hq)))
        _check(_lib().qmm_attn_prompt(t, q, k, v, o, n, hq, hkv, dim, seq_starts.data_ptr(), seq_starts.shape[0] - 1,
                                      dim ** -0.5 if scale is None else scale, place.stream.cuda_stream),
               "qmm_attn_prompt")
    return O


def qmm_attn_shared_workspace_bytes(n_seqs: int, prefix_len: int, own_cap: int, n_q_heads: int, n_kv_heads: int,
                                    head_dim: int) -> int:
    return int(_lib().qmm_attn_shared_workspace_bytes(int(n_seqs), int(prefix_len), int(own_cap), int(n_q_heads),
                                                      int(n_kv_heads), int(head_dim)))


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
    with _Place(stream, (("Q", Q), ("PK", PK), ("PV", PV), ("K", K), ("V", V), ("lengths", lengths), ("O", O),
                         ("workspace", workspace))) as place:
        if (PK is None) != (PV is None) or (K is None) != (V is None) or (K is None) != (lengths is None):
            raise ValueError("pass PK and PV together, and K, V and lengths together")
        if Q.dim() != 3 or (PK is not None and PK.dim() != 3) or (K is not None and K.dim() != 4):
            raise ValueError("Q must be [n_seqs][n_q_heads][head_dim], PK and PV [prefix_len][n_kv_heads][head_dim], "
                             "K and V [n_seqs][own_cap][n_kv_heads][head_dim]")
        n, hq, dim = Q.shape
        if PK is None and K is None:
            raise ValueError("pass a prefix, own caches or both")
        prefix, cap = (0 if PK is None else PK.shape[0]), (0 if K is None else K.shape[1])
        hkv = PK.shape[1] if PK is not None else K.shape[2]
        t = _type(Q, "Q", (QMM_T_F16, QMM_T_BF16))
        if O is None:
            O = place.empty((n, hq, dim), Q.dtype)
        q, o = _heads(Q, "Q", (n, hq, dim), Q.dtype), _heads(O, "O", (n, hq, dim), Q.dtype)
        pk = pv = k = v = None
        if PK is not None:
            pk, pv = _heads(PK, "PK", (prefix, hkv, dim), Q.dtype), _heads(PV, "PV", (prefix, hkv, dim), Q.dtype)
        if K is not None:
            k, v = _heads(K, "K", (n, cap, hkv, dim), Q.dtype), _heads(V, "V", (n, cap, hkv, dim), Q.dtype)
            _ints(lengths, "lengths", n)
        L = _lib()
        ws, ws_bytes, _keep = place.workspace(workspace, L.qmm_attn_shared_workspace_bytes(n, prefix, cap, hq, hkv, dim),
                                              "qmm_attn_shared_workspace_bytes")
        _check(L.qmm_attn_shared(t, q, pk, pv, prefix, k, v, cap, _ptr(lengths), o, n, hq, hkv, dim,
                                 dim ** -0.5 if scale is None else scale, ws, ws_bytes, place.stream.cuda_stream),
               "qmm_attn_shared")
    return O
