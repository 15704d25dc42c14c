"""Python binding of the prompt side of the LoopKV C ABI (include/loopkv_chunk.h).

Argument marshalling and checks only, as in loopkv.py.  Input rows may be
strided views (of one fused projection); outputs are contiguous.
"""

from __future__ import annotations

import ctypes

import torch

from .loopkv import KVCells, LoopKVError, library, loopkv_cells, loopkv_config


class loopkv_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class loopkv_rotary(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_positions", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_double)]


def _declare(lib):
    P, I32, VP = ctypes.POINTER, ctypes.c_int32, ctypes.c_void_p
    cell = [P(loopkv_config), P(loopkv_cells), I32, I32]
    rows, rotary = P(loopkv_rows), P(loopkv_rotary)
    sig = {
        "loopkv_norm_rope": [rotary, I32, I32, I32, rows, rows, VP, VP, I32, I32, VP, VP, VP, VP],
        "loopkv_rope_append": [*cell, rotary, rows, rows, rows, VP, VP, VP, I32, I32, VP, VP, VP],
        "loopkv_read_tokens": [*cell, VP, VP, VP, I32, I32, VP, VP, VP, VP],
        "loopkv_chunk_attention": [*cell, rows, rows, rows, VP, VP, VP, I32, I32, I32, ctypes.c_float, VP, VP, VP],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, args
    return lib


_lib = _declare(library())


def rope_table(max_positions: int, rotary_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [max_positions, rotary_dim]: the cosines, then the sines, of
    p * base^(-2 i / rotary_dim), with the angles in 64 bits (in 32 those of
    far positions lose their last digits)."""
    half = rotary_dim // 2
    freq = float(base) ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


class Rotary:
    """How a layer's queries and keys are normed and rotated.

    table    : CUDA fp32 [max_positions, rotary_dim] as from ``rope_table``, or
               None (no rotation); rotary_dim a multiple of 16, at most head_dim
    interleaved : pairs of neighbouring channels instead of the two halves
    q_weight, k_weight : CUDA bf16 [head_dim] of the norms for each head, or
               None (not normed)
    """

    def __init__(self, table=None, interleaved: bool = False, q_weight=None, k_weight=None, eps: float = 1e-6):
        if table is not None:
            _tensor(table, "table", torch.float32, 2)
            if not table.is_contiguous():
                raise ValueError("table must be contiguous")
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _tensor(w, name, torch.bfloat16, 1)
                if not w.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
        self.table, self.q_weight, self.k_weight = table, q_weight, k_weight
        self.interleaved, self.eps = bool(interleaved), float(eps)
        positions, dim = (0, 0) if table is None else table.shape
        self.struct = loopkv_rotary(_data(table), int(positions), int(dim), int(self.interleaved), _data(q_weight),
                                    _data(k_weight), self.eps)

    def _check(self, head_dim: int, device):
        for name, w in (("q_weight", self.q_weight), ("k_weight", self.k_weight)):
            if w is not None and w.shape[0] != head_dim:
                raise ValueError(f"{name} must have {head_dim} entries")
        for name, x in (("table", self.table), ("q_weight", self.q_weight), ("k_weight", self.k_weight)):
            if x is not None and x.device != device:
                raise ValueError(f"{name} is on {x.device}, the chunk on {device}")


def _data(t):
    return None if t is None else t.data_ptr()


def _tensor(t, what, dtype, dims):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{what} must have {dims} dimensions, got {tuple(t.shape)}")


def _rows(t, what, shape, device):
    """Rows bf16 [batch, tokens, heads, D], last dimension contiguous, others strided."""
    _tensor(t, what, torch.bfloat16, 4)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if t.stride(3) != 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    strides = [0 if n == 1 else s for n, s in zip(t.shape[:3], t.stride()[:3])]
    if t.numel() and (any(s % 8 for s in strides) or t.data_ptr() % 16):
        raise ValueError(f"{what} must be 16-byte aligned, with strides that are multiples of 8 elements")
    return loopkv_rows(t.data_ptr(), *strides)


def _ints(t, what, shape, device, optional=False):
    if t is None and optional:
        return None
    _tensor(t, what, torch.int32, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    return ctypes.c_void_p(t.data_ptr())


def _span(t):
    """First and one past the last byte that a tensor reaches."""
    if t.numel() == 0:
        return t.data_ptr(), t.data_ptr()
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _overlap(a, b):
    (a0, a1), (b0, b1) = _span(a), _span(b)
    return a0 < b1 and b0 < a1


def _output(out, what, shape, device, inputs, itself=None):
    """The contiguous output, zeros if not given; apart from every input but `itself` (in place)."""
    if out is None:
        return torch.zeros(shape, dtype=torch.bfloat16, device=device)
    _tensor(out, what, torch.bfloat16, len(shape))
    if tuple(out.shape) != tuple(shape) or not out.is_contiguous() or out.device != device:
        raise ValueError(f"{what} must be a contiguous {tuple(shape)} tensor on {device}")
    if out.data_ptr() % 16:
        raise ValueError(f"{what} must be 16-byte aligned")
    for name, x in inputs.items():
        if x is None or not _overlap(out, x):
            continue
        if name == itself and x.data_ptr() == out.data_ptr() and x.is_contiguous():
            continue
        raise ValueError(f"{what} overlaps {name}")
    return out


def _err(err_flag, device):
    if err_flag is None:
        return None
    _tensor(err_flag, "err_flag", torch.int32, err_flag.dim() if isinstance(err_flag, torch.Tensor) else 1)
    if err_flag.numel() < 1 or err_flag.device != device:
        raise ValueError(f"err_flag must be an int32 word on {device}")
    return ctypes.c_void_p(err_flag.data_ptr())


def _stream(stream, device):
    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError(f"the stream is on {s.device}, the tensors on {device}")
    return ctypes.c_void_p(s.cuda_stream)


def _cell_device(kv: KVCells, loop: int, layer: int):
    """Device of the storage that cell (loop, layer) reads or writes."""
    if not (0 <= loop < kv.num_loops and 0 <= layer < kv.num_layers):
        raise ValueError(f"no cell ({loop}, {layer}) in {kv.num_loops} loops of {kv.num_layers} layers")
    arena = kv.arenas[kv.source_cell(loop * kv.num_layers + layer)]
    if arena is None:
        raise ValueError(f"cell ({loop}, {layer}) has no storage")
    return arena.device


def _call(name, device, *args):
    with torch.cuda.device(device):
        st = getattr(_lib, name)(*args)
    if st:
        raise LoopKVError(st, name)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def loopkv_norm_rope(rotary: Rotary, q, k, start_pos, new_lens=None, q_out=None, k_out=None, err_flag=None,
                     stream=None):
    """Norms and rotation of a chunk's queries bf16 [B, T, H, D] and keys bf16
    [B, T, Hkv, D] (either may be None) at positions start_pos[b] + i in one
    pass; returns (q_out, k_out).  Rows from new_lens[b] on are left as they are
    (zeros in new outputs).  q_out may be q and k_out may be k, where contiguous."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k is required")
    _tensor(first, "q" if q is not None else "k", torch.bfloat16, 4)
    batch, tokens, _, dim = (int(x) for x in first.shape)
    dev = first.device
    rotary._check(dim, dev)
    heads = [0 if x is None or not isinstance(x, torch.Tensor) or x.dim() != 4 else int(x.shape[2]) for x in (q, k)]
    rows = [None if x is None else _rows(x, what, (batch, tokens, n, dim), dev)
            for x, what, n in ((q, "q", heads[0]), (k, "k", heads[1]))]
    ins = {"q": q, "k": k}
    if q is not None:
        q_out = _output(q_out, "q_out", q.shape, dev, ins, "q")
    if k is not None:
        k_out = _output(k_out, "k_out", k.shape, dev, ins, "k")
    if q is not None and k is not None and _overlap(q_out, k_out):
        raise ValueError("q_out overlaps k_out")
    _call("loopkv_norm_rope", dev, ctypes.byref(rotary.struct), dim, heads[0], heads[1], _ref(rows[0]), _ref(rows[1]),
          _ints(start_pos, "start_pos", (batch,), dev), _ints(new_lens, "new_lens", (batch,), dev, True), batch, tokens,
          _data(q_out) if q is not None else None, _data(k_out) if k is not None else None, _err(err_flag, dev),
          _stream(stream, dev))
    return (q_out if q is not None else None), (k_out if k is not None else None)


def loopkv_rope_append(kv: KVCells, loop: int, layer: int, rotary, q, k_new, v_new, block_table, start_pos,
                       new_lens=None, q_out=None, err_flag=None, stream=None):
    """Append a chunk's keys (normed and rotated; as they are if rotary is None)
    and values bf16 [B, T, Hkv, D] to a stored cell at positions start_pos[b] ..
    start_pos[b] + new_lens[b] - 1, and norm and rotate its queries bf16
    [B, T, H, D] (or None) in the same launch; returns q_out."""
    dev = _cell_device(kv, loop, layer)
    _tensor(k_new, "k_new", torch.bfloat16, 4)
    batch, tokens = int(k_new.shape[0]), int(k_new.shape[1])
    shape = (batch, tokens, kv.num_kv_heads, kv.head_dim)
    if rotary is not None:
        rotary._check(kv.head_dim, dev)
    elif q is not None:
        raise ValueError("q needs a rotary")
    kr, vr = _rows(k_new, "k_new", shape, dev), _rows(v_new, "v_new", shape, dev)
    qr = None
    if q is not None:
        qr = _rows(q, "q", (batch, tokens, kv.num_heads, kv.head_dim), dev)
        q_out = _output(q_out, "q_out", q.shape, dev, {"q": q, "k_new": k_new, "v_new": v_new}, "q")
    _call("loopkv_rope_append", dev, ctypes.byref(kv.cfg), ctypes.byref(kv.cells), loop, layer,
          None if rotary is None else ctypes.byref(rotary.struct), _ref(qr), ctypes.byref(kr), ctypes.byref(vr),
          _ints(block_table, "block_table", (batch, kv.max_blocks_per_seq), dev),
          _ints(start_pos, "start_pos", (batch,), dev), _ints(new_lens, "new_lens", (batch,), dev, True), batch, tokens,
          _data(q_out) if q is not None else None, _err(err_flag, dev), _stream(stream, dev))
    return q_out if q is not None else None


def loopkv_read_tokens(kv: KVCells, loop: int, layer: int, block_table, seq_lens, start_pos, num_tokens: int,
                       k_out=None, v_out=None, err_flag=None, stream=None):
    """Tokens start_pos[b] .. start_pos[b] + num_tokens - 1 of a cell that holds
    seq_lens[b], as bf16 values [B, num_tokens, Hkv, D]; returns (k_out, v_out).
    Rows of tokens that are not there are left as they are (zeros in new
    outputs)."""
    dev = _cell_device(kv, loop, layer)
    _tensor(start_pos, "start_pos", torch.int32, 1)
    batch, num_tokens = int(start_pos.shape[0]), int(num_tokens)
    shape = (batch, max(num_tokens, 0), kv.num_kv_heads, kv.head_dim)
    outs = [_output(o, what, shape, dev, {}) for o, what in ((k_out, "k_out"), (v_out, "v_out"))]
    if _overlap(*outs):
        raise ValueError("k_out overlaps v_out")
    _call("loopkv_read_tokens", dev, ctypes.byref(kv.cfg), ctypes.byref(kv.cells), loop, layer,
          _ints(block_table, "block_table", (batch, kv.max_blocks_per_seq), dev),
          _ints(seq_lens, "seq_lens", (batch,), dev), _ints(start_pos, "start_pos", (batch,), dev), batch, num_tokens,
          _data(outs[0]), _data(outs[1]), _err(err_flag, dev), _stream(stream, dev))
    return outs[0], outs[1]


def loopkv_chunk_attention(kv: KVCells, loop: int, layer: int, q, block_table, start_pos, new_lens=None,
                           sm_scale: float = 1.0, out=None, max_seq_len: int = 0, k_cur=None, v_cur=None,
                           err_flag=None, stream=None):
    """Attention of a chunk's queries bf16 [B, T, H, D] at positions start_pos[b]
    + i over cell (loop, layer); returns out bf16 [B, T, H, D].  Without k_cur
    and v_cur a query sees the stored tokens up to its own position; with them
    (bf16 [B, T, Hkv, D]) the start_pos[b] stored tokens and the chunk's exact
    rows up to its own.  Rows from new_lens[b] on are left as they are (zeros in
    a new output)."""
    dev = _cell_device(kv, loop, layer)
    _tensor(q, "q", torch.bfloat16, 4)
    batch, tokens = int(q.shape[0]), int(q.shape[1])
    qr = _rows(q, "q", (batch, tokens, kv.num_heads, kv.head_dim), dev)
    if (k_cur is None) != (v_cur is None):
        raise ValueError("k_cur and v_cur come together")
    kr = vr = None
    if k_cur is not None:
        shape = (batch, tokens, kv.num_kv_heads, kv.head_dim)
        kr, vr = _rows(k_cur, "k_cur", shape, dev), _rows(v_cur, "v_cur", shape, dev)
    if out is None and new_lens is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)  # every row is written
    out = _output(out, "out", q.shape, dev, {"q": q, "k_cur": k_cur, "v_cur": v_cur})
    _call("loopkv_chunk_attention", dev, ctypes.byref(kv.cfg), ctypes.byref(kv.cells), loop, layer, ctypes.byref(qr),
          _ref(kr), _ref(vr), _ints(block_table, "block_table", (batch, kv.max_blocks_per_seq), dev),
          _ints(start_pos, "start_pos", (batch,), dev), _ints(new_lens, "new_lens", (batch,), dev, True), batch, tokens,
          int(max_seq_len), float(sm_scale), _data(out), _err(err_flag, dev), _stream(stream, dev))
    return out
