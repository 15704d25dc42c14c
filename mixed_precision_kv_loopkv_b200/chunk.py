"""Python binding of the prompt side of the LoopKV C ABI (include/loopkv_chunk.h).

Argument marshalling and checks only, as in loopkv.py.  Input rows may be
strided views (of one fused projection); outputs are contiguous.
"""

from __future__ import annotations

import ctypes

import torch

from .loopkv import KVCells, LoopKVError, library, loopkv_cells, loopkv_config


_BF16, _INT32 = torch.bfloat16, torch.int32

try:  # the handle alone: a Stream object takes a microsecond to make
    from torch._C import _cuda_getCurrentRawStream as _current_stream
except ImportError:
    def _current_stream(dev):
        return torch.cuda.current_stream(dev).cuda_stream


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
        parts = {"table": (table, torch.float32, 2), "q_weight": (q_weight, torch.bfloat16, 1),
                 "k_weight": (k_weight, torch.bfloat16, 1)}
        devices, self._dims = set(), {}
        for name, (x, dtype, dims) in parts.items():
            if x is None:
                continue
            if not isinstance(x, torch.Tensor) or not x.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if x.dtype != dtype or x.dim() != dims or not x.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of {dims} dimensions")
            devices.add(x.get_device())
            if dims == 1:
                self._dims[name] = int(x.shape[0])
        if len(devices) > 1:
            raise ValueError("the table and the weights are on different devices")
        self._device = devices.pop() if devices else None
        self.table, self.q_weight, self.k_weight = table, q_weight, k_weight
        self.interleaved, self.eps = bool(interleaved), float(eps)
        positions, dim = (0, 0) if table is None else table.shape
        self.struct = loopkv_rotary(_data(table), int(positions), int(dim), int(self.interleaved), _data(q_weight),
                                    _data(k_weight), self.eps)

    def _check(self, head_dim: int, dev: int):
        if self._device is not None and self._device != dev:
            raise ValueError(f"the rotary is on cuda:{self._device}, the chunk on cuda:{dev}")
        for name, n in self._dims.items():
            if n != head_dim:
                raise ValueError(f"{name} must have {head_dim} entries")


# The checks below run at every call, beside kernels of a few microseconds: one
# comparison of what is expected each, and the reason worked out only when it fails.


def _data(t):
    return None if t is None else t.data_ptr()


def _device_of(t, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.get_device()


def _refuse(t, what, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{what} is on {t.device}, expected cuda:{dev}")


def _is(t, dtype, shape, dev):
    try:
        return t.dtype is dtype and t.get_device() == dev and t.shape == shape
    except AttributeError:  # no tensor
        return False


def _rows(t, what, shape, dev):
    """Rows bf16 [batch, tokens, heads, D], last dimension contiguous, others
    strided: the C struct, and the first and one past the last byte they reach."""
    if not _is(t, _BF16, shape, dev):
        _refuse(t, what, _BF16, shape, dev)
    b, n, h, d = shape
    sb, st, sh, sd = t.stride()
    ptr = t.data_ptr()
    if (sb | st | sh) & 7 or ptr & 15 or sd != 1:
        # the stride of a dimension of one says nothing
        sb, st, sh = (0 if k == 1 else x for k, x in zip(shape, (sb, st, sh)))
        if ((sb | st | sh) & 7 or ptr & 15 or sd != 1) and t.numel():
            raise ValueError(f"{what} must be contiguous in its last dimension, 16-byte aligned, with strides that are "
                             "multiples of 8 elements")
    return loopkv_rows(ptr, sb, st, sh), ptr, ptr + 2 * ((b - 1) * sb + (n - 1) * st + (h - 1) * sh + d)


def _ints(t, what, shape, dev):
    if not _is(t, _INT32, shape, dev):
        _refuse(t, what, _INT32, shape, dev)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _new(shape, dev, stream, fill=True):
    """A new output, made (and filled with zeros) on the stream of the call."""
    make = torch.zeros if fill else torch.empty
    if stream is None:
        return make(shape, dtype=torch.bfloat16, device=f"cuda:{dev}")
    with torch.cuda.stream(stream):
        return make(shape, dtype=torch.bfloat16, device=f"cuda:{dev}")


def _output(out, what, shape, dev, stream, inputs=(), itself=None):
    """The contiguous output, zeros if not given.  It must lie apart from every
    input (name, tensor, its rows) but ``itself``, which it may be (in place)."""
    if out is None:
        return _new(shape, dev, stream)
    if not _is(out, _BF16, shape, dev):
        _refuse(out, what, _BF16, shape, dev)
    ptr = out.data_ptr()
    if not out.is_contiguous() or ptr & 15:
        raise ValueError(f"{what} must be contiguous and 16-byte aligned")
    end = ptr + 2 * out.numel()
    for name, x, rows in inputs:
        if rows[1] < end and ptr < rows[2]:
            if not (name == itself and rows[1] == ptr and x.is_contiguous()):
                raise ValueError(f"{what} overlaps {name}")
    return out


def _apart(a, b):
    """Whether two contiguous outputs share no byte."""
    return a.data_ptr() + 2 * a.numel() <= b.data_ptr() or b.data_ptr() + 2 * b.numel() <= a.data_ptr()


def _err(err_flag, dev):
    if err_flag is None:
        return None
    if not isinstance(err_flag, torch.Tensor) or err_flag.dtype != torch.int32 or err_flag.numel() < 1 \
            or err_flag.get_device() != dev:
        raise ValueError(f"err_flag must be an int32 word on cuda:{dev}")
    return err_flag.data_ptr()


def _cell_device(kv: KVCells, loop: int, layer: int):
    """Device of the storage that cell (loop, layer) reads or writes."""
    if not (0 <= loop < kv.num_loops and 0 <= layer < kv.num_layers):
        raise ValueError(f"no cell ({loop}, {layer}) in {kv.num_loops} loops of {kv.num_layers} layers")
    arena = kv.arenas[kv.source_cell(loop * kv.num_layers + layer)]
    if arena is None:
        raise ValueError(f"cell ({loop}, {layer}) has no storage")
    dev = arena.get_device()
    if dev < 0:
        raise ValueError("the cell's storage must be on a CUDA device")
    return dev


def _call(fn, name, dev, stream, *args):
    """Call on the tensors' device, whichever is current, on its current stream
    unless another of its streams is given."""
    if stream is None:
        handle = _current_stream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        handle = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st:
        raise LoopKVError(st, name)


def loopkv_norm_rope(rotary: Rotary, q, k, start_pos, new_lens=None, q_out=None, k_out=None, err_flag=None,
                     stream=None):
    """Norms and rotation of a chunk's queries bf16 [B, T, H, D] and keys bf16
    [B, T, Hkv, D] (either may be None) at positions start_pos[b] + i in one
    pass; returns (q_out, k_out).  Rows from new_lens[b] on are left as they are
    (zeros in new outputs).  q_out may be q and k_out may be k, where contiguous."""
    first, what = (q, "q") if q is not None else (k, "k")
    if first is None:
        raise ValueError("q or k is required")
    dev = _device_of(first, what)
    if first.dim() != 4:
        raise ValueError(f"{what} must be [batch, tokens, heads, head_dim]")
    batch, tokens, _, dim = first.shape
    rotary._check(dim, dev)
    heads, kv_heads, qr, kr, ins = 0, 0, None, None, []
    if q is not None:
        heads = q.shape[2]
        qr = _rows(q, "q", (batch, tokens, heads, dim), dev)
        ins.append(("q", q, qr))
    if k is not None:
        kv_heads = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
        kr = _rows(k, "k", (batch, tokens, kv_heads, dim), dev)
        ins.append(("k", k, kr))
    q_out = _output(q_out, "q_out", q.shape, dev, stream, ins, "q") if qr else None
    k_out = _output(k_out, "k_out", k.shape, dev, stream, ins, "k") if kr else None
    if qr and kr and not _apart(q_out, k_out):
        raise ValueError("q_out overlaps k_out")
    lens = None if new_lens is None else _ints(new_lens, "new_lens", (batch,), dev)
    _call(_lib.loopkv_norm_rope, "loopkv_norm_rope", dev, stream, rotary.struct, dim, heads, kv_heads,
          qr and qr[0], kr and kr[0], _ints(start_pos, "start_pos", (batch,), dev), lens, batch, tokens, _data(q_out),
          _data(k_out), _err(err_flag, dev))
    return q_out, k_out


def loopkv_rope_append(kv: KVCells, loop: int, layer: int, rotary, q, k_new, v_new, block_table, start_pos,
                       new_lens=None, q_out=None, err_flag=None, stream=None):
    """Append a chunk's keys (normed and rotated; as they are if rotary is None)
    and values bf16 [B, T, Hkv, D] to a stored cell at positions start_pos[b] ..
    start_pos[b] + new_lens[b] - 1, and norm and rotate its queries bf16
    [B, T, H, D] (or None) in the same launch; returns q_out (new: zeros where
    there is no row).  start_pos is what the cell holds; a 4-bit or 2-bit cell
    can go back to the last multiple of 32 tokens and no further, so drafted
    tokens are appended when they are accepted (LoopedChunkStep.store)."""
    dev = _cell_device(kv, loop, layer)
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 4:
        raise ValueError("k_new must be [batch, tokens, heads, head_dim]")
    batch, tokens = k_new.shape[:2]
    shape = (batch, tokens, kv.num_kv_heads, kv.head_dim)
    if rotary is not None:
        rotary._check(kv.head_dim, dev)
    elif q is not None:
        raise ValueError("q needs a rotary")
    kr, vr, qr = _rows(k_new, "k_new", shape, dev), _rows(v_new, "v_new", shape, dev), None
    if q is not None:
        shape = (batch, tokens, kv.num_heads, kv.head_dim)
        qr = _rows(q, "q", shape, dev)
        q_out = _output(q_out, "q_out", shape, dev, stream, (("q", q, qr), ("k_new", k_new, kr), ("v_new", v_new, vr)), "q")
    else:
        q_out = None
    lens = None if new_lens is None else _ints(new_lens, "new_lens", (batch,), dev)
    _call(_lib.loopkv_rope_append, "loopkv_rope_append", dev, stream, kv.cfg, kv.cells, loop, layer,
          rotary and rotary.struct, qr and qr[0], kr[0], vr[0],
          _ints(block_table, "block_table", (batch, kv.max_blocks_per_seq), dev),
          _ints(start_pos, "start_pos", (batch,), dev), lens, batch, tokens, _data(q_out), _err(err_flag, dev))
    return q_out


def loopkv_read_tokens(kv: KVCells, loop: int, layer: int, block_table, seq_lens, start_pos, num_tokens: int,
                       k_out=None, v_out=None, err_flag=None, stream=None):
    """Tokens start_pos[b] .. start_pos[b] + num_tokens - 1 of a cell that holds
    seq_lens[b], as bf16 values [B, num_tokens, Hkv, D]; returns (k_out, v_out).
    Rows of tokens that are not there are left as they are (zeros in new
    outputs)."""
    dev = _cell_device(kv, loop, layer)
    num_tokens = int(num_tokens)
    if not isinstance(start_pos, torch.Tensor) or start_pos.dim() != 1 or num_tokens < 0:
        raise ValueError("start_pos must be [batch], num_tokens not negative")
    batch = start_pos.shape[0]
    shape = (batch, num_tokens, kv.num_kv_heads, kv.head_dim)
    k_out, v_out = _output(k_out, "k_out", shape, dev, stream), _output(v_out, "v_out", shape, dev, stream)
    if not _apart(k_out, v_out):
        raise ValueError("k_out overlaps v_out")
    _call(_lib.loopkv_read_tokens, "loopkv_read_tokens", dev, stream, kv.cfg, kv.cells, loop, layer,
          _ints(block_table, "block_table", (batch, kv.max_blocks_per_seq), dev),
          _ints(seq_lens, "seq_lens", (batch,), dev), _ints(start_pos, "start_pos", (batch,), dev), batch, num_tokens,
          k_out.data_ptr(), v_out.data_ptr(), _err(err_flag, dev))
    return k_out, v_out


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
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [batch, tokens, heads, head_dim]")
    batch, tokens = q.shape[:2]
    shape = (batch, tokens, kv.num_heads, kv.head_dim)
    qr, kr, vr = _rows(q, "q", shape, dev), None, None
    ins = [("q", q, qr)]
    if (k_cur is None) != (v_cur is None):
        raise ValueError("k_cur and v_cur come together")
    if k_cur is not None:
        rows = (batch, tokens, kv.num_kv_heads, kv.head_dim)
        kr, vr = _rows(k_cur, "k_cur", rows, dev), _rows(v_cur, "v_cur", rows, dev)
        ins += [("k_cur", k_cur, kr), ("v_cur", v_cur, vr)]
    if out is None and new_lens is None:
        out = _new(shape, dev, stream, fill=False)  # every row is written
    else:
        out = _output(out, "out", shape, dev, stream, ins)
    lens = None if new_lens is None else _ints(new_lens, "new_lens", (batch,), dev)
    _call(_lib.loopkv_chunk_attention, "loopkv_chunk_attention", dev, stream, kv.cfg, kv.cells, loop, layer, qr[0],
          kr and kr[0], vr and vr[0], _ints(block_table, "block_table", (batch, kv.max_blocks_per_seq), dev),
          _ints(start_pos, "start_pos", (batch,), dev), lens, batch, tokens, int(max_seq_len), float(sm_scale),
          out.data_ptr(), _err(err_flag, dev))
    return out
