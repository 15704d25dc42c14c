"""Plain CPU oracle of the prompt side: norms, rotation and chunk attention.

The norm and rotation follow the definition step by step in numpy float32 (one
rounded operation each, the mean of the squares in 64 bits); the attention is
64-bit throughout, on the values that a stored cell's tokens stand for.
"""

from __future__ import annotations

import numpy as np

from .loopkv_oracle import StoredSequence, bf16_round


def rope_angles(positions: int, rotary_dim: int, base: float = 10000.0) -> np.ndarray:
    """fp32 [positions, rotary_dim]: cosines, then sines, from 64-bit angles."""
    half = rotary_dim // 2
    freq = float(base) ** (-np.arange(half, dtype=np.float64) / half)
    angle = np.arange(positions, dtype=np.float64)[:, None] * freq
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)


def norm_rope(x, positions, table=None, interleaved: bool = False, weight=None, eps: float = 1e-6) -> np.ndarray:
    """Rows x fp32[tokens, heads, D] (bf16 values) at positions int[tokens]; bf16 values fp32."""
    x = np.asarray(x, np.float32)
    if weight is not None:
        mean = (x.astype(np.float64) ** 2).sum(-1, keepdims=True) / x.shape[-1]
        r = (1.0 / np.sqrt(mean + eps)).astype(np.float32)
        x = (x * r) * np.asarray(weight, np.float32)
    y = x.copy()
    if table is not None:
        rot = table.shape[1]
        half = rot // 2
        row = np.asarray(table, np.float32)[np.asarray(positions)][:, None, :]
        cos, sin = row[..., :half], row[..., half:]
        first = np.arange(0, rot, 2) if interleaved else np.arange(half)
        second = first + (1 if interleaved else half)
        a, b = x[..., first], x[..., second]
        y[..., first] = a * cos - b * sin
        y[..., second] = b * cos + a * sin
    return bf16_round(y)


def stored_values(kind: str, k, v):
    """fp64 keys and values that a cell holding the tokens k, v stands for."""
    seq = StoredSequence(kind, k, v)
    if kind == "bf16":
        return seq.k_exact.astype(np.float64), seq.v_exact.astype(np.float64)
    return seq.qk.dequant(), seq.qv.dequant_full()


def chunk_attend(q, k_hat, v_hat, last, sm_scale: float):
    """Attention of rows q fp64[rows, D]; row i sees keys 0 .. last[i] (none: zeros).

    Returns (out fp64[rows, D], slack fp64[rows, D]).  slack bounds what 16-bit
    tensor-core operands may move the result by, to first order: a key or value
    entry off by u = 2^-11 of itself, a weight by u, a weight below 2^-14 by
    2^-25 of the largest, and fp32 sums.  With d_j = (u + D 2^-23) sm sum_c |q_c k_jc|
    the weight p_j is off by at most p_j (d_j + sum_i p_i d_i), so
      slack_c = sum_j p_j |v_jc| (d_j + sum_i p_i d_i + 2 u + 2^-16) + 2^-25 sum_j |v_jc|,
    times 1.05 for the terms of second order, plus the output's own rounding 2^-8 |out_c|
    (half of a bf16 step relative to the value).
    """
    q, k_hat, v_hat = (np.asarray(x, np.float64) for x in (q, k_hat, v_hat))
    rows, d = q.shape
    out, slack = np.zeros((rows, d)), np.zeros((rows, d))
    u = 2.0**-11
    for i in range(rows):
        n = int(last[i]) + 1
        if n <= 0:
            continue
        s = sm_scale * (k_hat[:n] @ q[i])
        e = np.exp(s - s.max())
        p = e / e.sum()
        out[i] = p @ v_hat[:n]
        dj = (u + d * 2.0**-23) * abs(sm_scale) * (np.abs(k_hat[:n]) @ np.abs(q[i]))
        w = p * (dj + p @ dj + 2 * u + 2.0**-16)
        slack[i] = 1.05 * (w @ np.abs(v_hat[:n]) + 2.0**-25 * np.abs(v_hat[:n]).sum(0)) + 2.0**-8 * np.abs(out[i])
    return out, slack
