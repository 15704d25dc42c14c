"""Refusals of the prompt-side entry points, and what their host code computes
(no kernel is launched: argument errors return before any CUDA call)."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import oracle as O
from oracle import chunk_oracle as CO
from test_abi import BF16, Q2, Q4, REUSE, _cells, _cfg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x20000


@pytest.fixture(scope="module")
def m():
    import mixed_precision_kv_loopkv_b200 as pkg
    return pkg


@pytest.fixture(scope="module")
def c():
    from mixed_precision_kv_loopkv_b200 import chunk
    return chunk


def test_header_functions_are_exported(m):
    text = open(os.path.join(ROOT, "include", "loopkv_chunk.h")).read()
    names = re.findall(r"LOOPKV_API\s+[\w\s\*]+?\b(loopkv_\w+)\s*\(", text)
    assert sorted(names) == ["loopkv_chunk_attention", "loopkv_norm_rope", "loopkv_read_tokens", "loopkv_rope_append"]
    lib = ctypes.CDLL(m.LIB_PATH)
    for name in names:
        assert hasattr(lib, name) and callable(getattr(m, name)), name


def _rows(c, data=FAKE, b=4096, t=1024, h=128):
    return c.loopkv_rows(data, b, t, h)


def _rotary(c, cos_sin=FAKE, positions=64, dim=64, interleaved=0, qw=None, kw=None, eps=1e-6):
    return c.loopkv_rotary(cos_sin, positions, dim, interleaved, qw, kw, eps)


def _ref(x):
    return None if x is None else ctypes.byref(x)


OK_ROWS = "rows"


def _norm_rope(m, c, rotary=None, dim=128, heads=2, kv_heads=2, q=OK_ROWS, k=OK_ROWS, start=FAKE, batch=1, tokens=1,
               q_out=FAKE, k_out=FAKE):
    q, k = (_rows(c) if x is OK_ROWS else x for x in (q, k))
    rotary = _rotary(c) if rotary is None else rotary
    return m.library().loopkv_norm_rope(_ref(rotary), dim, heads, kv_heads, _ref(q), _ref(k), start, None, batch, tokens,
                                        q_out, k_out, None, None)


def _append(m, c, cfg, cells, rotary="yes", loop=0, layer=0, q=OK_ROWS, k=OK_ROWS, v=OK_ROWS, table=FAKE, start=FAKE,
            batch=1, tokens=1, q_out=FAKE):
    q, k, v = (_rows(c) if x is OK_ROWS else x for x in (q, k, v))
    rotary = _rotary(c) if rotary == "yes" else rotary
    return m.library().loopkv_rope_append(_ref(cfg), _ref(cells), loop, layer, _ref(rotary), _ref(q), _ref(k), _ref(v),
                                          table, start, None, batch, tokens, q_out, None, None)


def _read(m, cfg, cells, loop=0, layer=0, table=FAKE, lens=FAKE, start=FAKE, batch=1, tokens=1, k_out=FAKE, v_out=FAKE):
    return m.library().loopkv_read_tokens(_ref(cfg), _ref(cells), loop, layer, table, lens, start, batch, tokens, k_out,
                                          v_out, None, None)


def _attend(m, c, cfg, cells, loop=0, layer=0, q=OK_ROWS, k=None, v=None, table=FAKE, start=FAKE, batch=1, tokens=1,
            max_seq_len=0, sm_scale=1.0, out=FAKE):
    q = _rows(c) if q is OK_ROWS else q
    return m.library().loopkv_chunk_attention(_ref(cfg), _ref(cells), loop, layer, _ref(q), _ref(k), _ref(v), table,
                                              start, None, batch, tokens, max_seq_len, sm_scale, out, None, None)


def test_bad_rows_are_refused(m, c):
    cfg, cells = _cfg(m, [Q4], 1, 1), _cells(m, 1)
    for bad in (_rows(c, data=None), _rows(c, data=FAKE + 2), _rows(c, t=1020), _rows(c, h=4), _rows(c, b=-8)):
        assert _norm_rope(m, c, q=bad) == 1
        assert _norm_rope(m, c, k=bad) == 1
        for name in "qkv":
            assert _append(m, c, cfg, cells, **{name: bad}) == 1
        assert _attend(m, c, cfg, cells, q=bad) == 1
        assert _attend(m, c, cfg, cells, k=bad, v=_rows(c)) == 1
        assert _attend(m, c, cfg, cells, k=_rows(c), v=bad) == 1


def test_bad_rotary_is_refused(m, c):
    cfg, cells = _cfg(m, [Q4], 1, 1), _cells(m, 1)
    nan = float("nan")
    for kw in (dict(dim=8), dict(dim=72), dict(dim=144), dict(dim=0), dict(positions=0), dict(cos_sin=FAKE + 4),
               dict(interleaved=2), dict(qw=FAKE + 2), dict(kw=FAKE + 2), dict(kw=FAKE, eps=-1e-6),
               dict(kw=FAKE, eps=nan), dict(kw=FAKE, eps=0.0), dict(qw=FAKE, eps=float("inf"))):
        assert _norm_rope(m, c, rotary=_rotary(c, **kw)) == 1, kw
        assert _append(m, c, cfg, cells, rotary=_rotary(c, **kw)) == 1, kw
    assert _append(m, c, cfg, cells, rotary=None) == 1  # queries need a rotary


def test_norm_rope_refusals(m, c):
    assert _norm_rope(m, c, dim=96) == 3
    assert _norm_rope(m, c, q=None, k=None) == 1
    assert _norm_rope(m, c, heads=0) == 1
    assert _norm_rope(m, c, kv_heads=-1) == 1
    assert _norm_rope(m, c, batch=-1) == 1
    assert _norm_rope(m, c, tokens=-1) == 1
    assert _norm_rope(m, c, start=None) == 1
    assert _norm_rope(m, c, q_out=None) == 1
    assert _norm_rope(m, c, k_out=FAKE + 8) == 1
    assert _norm_rope(m, c, batch=1 << 16, tokens=1 << 14) == 3      # 2^32 rows
    assert _norm_rope(m, c, batch=0) == 0 and _norm_rope(m, c, tokens=0) == 0


def test_append_refusals(m, c):
    cfg, cells = _cfg(m, [Q4], 1, 1), _cells(m, 1)
    assert _append(m, c, cfg, cells, layer=1) == 1
    assert _append(m, c, cfg, cells, batch=3) == 1
    assert _append(m, c, cfg, cells, tokens=-1) == 1
    assert _append(m, c, cfg, cells, k=None) == 1
    assert _append(m, c, cfg, cells, table=None) == 1
    assert _append(m, c, cfg, cells, q_out=None) == 1
    assert _append(m, c, cfg, cells, batch=0) == 0 and _append(m, c, cfg, cells, tokens=0) == 0
    assert _append(m, c, _cfg(m, [REUSE, Q4], 2, 1), _cells(m, 2)) == 1       # a reuse cell stores nothing
    assert _append(m, c, _cfg(m, [Q4, REUSE], 2, 1), _cells(m, 2)) == 2
    assert _append(m, c, _cfg(m, [Q4], 1, 1, head_dim=96), cells) == 3


def test_read_refusals(m):
    cfg, cells = _cfg(m, [Q4], 1, 1), _cells(m, 1)
    assert _read(m, cfg, cells, loop=1) == 1
    assert _read(m, cfg, cells, batch=3) == 1
    assert _read(m, cfg, cells, tokens=-1) == 1
    assert _read(m, cfg, cells, lens=None) == 1
    assert _read(m, cfg, cells, k_out=None, v_out=None) == 1
    assert _read(m, cfg, cells, k_out=FAKE + 2) == 1
    assert _read(m, cfg, cells, batch=0) == 0 and _read(m, cfg, cells, tokens=0) == 0
    assert _read(m, _cfg(m, [Q4, 9], 1, 2), _cells(m, 2)) == 2


def test_attention_refusals(m, c):
    cfg, cells = _cfg(m, [Q4, Q2, REUSE, BF16], 1, 4), _cells(m, 4)
    assert _attend(m, c, cfg, cells) == 2                                     # a reuse cell in the final loop
    cfg, cells = _cfg(m, [Q4], 1, 1), _cells(m, 1)
    assert _attend(m, c, cfg, cells, batch=3) == 1
    assert _attend(m, c, cfg, cells, tokens=-1) == 1
    assert _attend(m, c, cfg, cells, max_seq_len=65) == 1                     # beyond the block table
    assert _attend(m, c, cfg, cells, max_seq_len=-1) == 1
    assert _attend(m, c, cfg, cells, sm_scale=float("inf")) == 1
    assert _attend(m, c, cfg, cells, k=_rows(c)) == 1                         # both rows or neither
    assert _attend(m, c, cfg, cells, q=None) == 1
    assert _attend(m, c, cfg, cells, out=None) == 1
    assert _attend(m, c, cfg, cells, out=FAKE + 2) == 1
    assert _attend(m, c, cfg, cells, start=None) == 1
    assert _attend(m, c, cfg, cells, batch=0) == 0 and _attend(m, c, cfg, cells, tokens=0) == 0
    assert _attend(m, c, _cfg(m, [Q4], 1, 1, num_heads=6, num_kv_heads=2), cells) == 3
    empty = _cells(m, 1)
    empty._keep[0][0] = None
    assert _attend(m, c, cfg, empty) == 1 and _read(m, cfg, empty) == 1 and _append(m, c, cfg, empty) == 1


def test_binding_refuses_host_tensors(m, c):
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        m.loopkv_norm_rope(m.Rotary(), x, None, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        m.Rotary(m.rope_table(8, 64, device="cpu"))


@pytest.mark.parametrize("rot", [16, 48, 64])
def test_rope_table_agrees_with_oracle(m, rot):
    got = m.rope_table(5000, rot, device="cpu").numpy()
    want = CO.rope_angles(5000, rot)
    # two libraries' 64-bit cosines, each within 2^-50 of the true one, rounded once to fp32
    assert got.shape == want.shape and np.max(np.abs(got.astype(np.float64) - want)) <= 2.0**-24


def test_oracle_rotation_keeps_lengths_and_relative_angles():
    """The rotation is orthogonal, and the product of two rotated rows depends on
    the distance of their positions alone (pinned without the kernel)."""
    rng = np.random.default_rng(0)
    for interleaved in (False, True):
        table = CO.rope_angles(64, 32).astype(np.float64)
        x = rng.standard_normal((1, 1, 32))
        y = rng.standard_normal((1, 1, 32))

        def turn(v, p):
            half = 16
            first = np.arange(0, 32, 2) if interleaved else np.arange(half)
            second = first + (1 if interleaved else half)
            c, s = table[p, :half], table[p, half:]
            o = v.copy()
            o[..., first], o[..., second] = v[..., first] * c - v[..., second] * s, v[..., second] * c + v[..., first] * s
            return o
        a = float((turn(x, 9) * turn(y, 4)).sum())
        b = float((turn(x, 45) * turn(y, 40)).sum())
        assert abs(a - b) < 1e-5
        xb = O.bf16_round(x.astype(np.float32))
        got = CO.norm_rope(xb, [9], table.astype(np.float32), interleaved)
        assert np.max(np.abs(got - turn(xb.astype(np.float64), 9))) <= 2.0**-8 * np.max(np.abs(got)) * 1.01


def test_oracle_chunk_of_one_is_decode():
    """A chunk of one token over n stored ones is the decode oracle at tau = 0."""
    rng = np.random.default_rng(1)
    k, v = (O.bf16_round(rng.standard_normal((70, 64)).astype(np.float32)) for _ in "kv")
    q = O.bf16_round(rng.standard_normal(64).astype(np.float32))
    for kind in ("q4", "q2", "bf16"):
        want, _, _ = O.StoredSequence(kind, k, v).attend(q, 0.0, 0.3)
        kh, vh = CO.stored_values(kind, k, v)
        got, slack = CO.chunk_attend(q[None], kh, vh, [69], 0.3)
        assert np.max(np.abs(got[0] - want)) < 1e-12 and np.all(slack > 0)
    empty, _ = CO.chunk_attend(q[None], k[:0], v[:0], [-1], 1.0)
    assert not empty.any()


def test_capacity_beyond_31_bits_is_unsupported(m, c):
    cfg, cells = _cfg(m, [Q4], 1, 1, max_blocks_per_seq=1 << 27), _cells(m, 1)
    assert _append(m, c, cfg, cells) == 3 and _read(m, cfg, cells) == 3 and _attend(m, c, cfg, cells) == 3


def test_scale_that_overflows_is_invalid(m, c):
    assert _attend(m, c, _cfg(m, [Q4], 1, 1), _cells(m, 1), sm_scale=3e38) == 1


def test_build_refuses_other_register_counts():
    """The register split of the 256-row kernels is compared with what the compiler
    used, when the library is built and not when a user calls it."""
    from mixed_precision_kv_loopkv_b200 import build
    source = "chunk_attention.cu"

    def report(*kernels):
        return "".join(f"ptxas info    : Compiling entry function '{name}' for 'sm_100a'\nptxas info    : Function properties "
                       f"for {name}\n    0 bytes stack frame\nptxas info    : Used {regs} registers, used 1 barriers\n"
                       for name, regs in kernels)

    good = [("_ZN6loopkv19chunk_tensor_kernelILi0ELi128ELi2EEEvNS", 96), ("_ZN6loopkv19chunk_tensor_kernelILi3ELi64ELi2EEEvNS", 96)]
    others = [("_ZN6loopkv19chunk_tensor_kernelILi0ELi128ELi1EEEvNS", 127), ("_ZN6loopkv16chunk_few_kernelILi0ELi128ELi12EEEvNS", 168)]
    assert build.check_registers(source, report(others[0], *good, others[1])) == 2
    assert build.check_registers("append.cu", "") == 0
    for bad in (report(good[0], (good[1][0], 88)), report((good[0][0], 104), good[1]), report(*others), ""):
        with pytest.raises(RuntimeError):
            build.check_registers(source, bad)


def test_polynomial_exponential():
    """The cubic of the softmax' FMA units: 7.5e-5 of 2^x at the most (its steps in
    fp32, each multiply-add rounded once), over every fraction and many exponents."""
    text = open(os.path.join(ROOT, "mixed_precision_kv_loopkv_b200", "csrc", "chunk_tensor.cuh")).read()
    body = text[text.index("void poly_exp2("):]
    body = body[:body.index("\n}\n")]
    c3, c2, c1, c0 = (np.float32(x) for x in re.findall(r"pack2\((\d\.\d+e-\d+)f, \1f\)", body))
    x = np.concatenate([np.linspace(-126, 100, 400_001), np.linspace(-1, 1, 400_001)]).astype(np.float32)
    magic = np.float32(12582912.0)
    n = (x + magic) - magic

    def fma(a, b, c):
        return (a.astype(np.float64) * b + np.float64(c)).astype(np.float32)   # exact product, one rounding to 53, one to 24 bits

    f = (x.astype(np.float64) - n).astype(np.float32)
    assert np.abs(f).max() <= 0.5
    y = fma(fma(fma(f, c3, c2), f, c1), f, c0)
    got = np.ldexp(y.astype(np.float64), n.astype(np.int64))
    rel = np.abs(got / np.exp2(x.astype(np.float64)) - 1)
    assert 7e-5 < rel.max() < 7.6e-5
