"""Chunk attention over numbers of far-apart and of extreme sizes: a row's
precision follows what it sees and weighs."""

import numpy as np
import pytest
import torch

from loopkv_testlib import seeded_bf16
from oracle import chunk_oracle as CO
from test_gpu_chunk import cell_for, host, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mixed_precision_kv_loopkv_b200 as pkg
    return pkg


def block_tops(vh, n, size):
    """The largest absolute value of each token's block of `size` tokens, over the n
    stored tokens and, counted anew, over the current ones."""
    top = np.zeros(vh.shape[0])
    for lo, hi in ((0, n), (n, vh.shape[0])):
        for t in range(lo, hi, size):
            top[t: min(t + size, hi)] = np.abs(vh[t: min(t + size, hi)]).max()
    return top


def attend_seen(q, kh, vh, last, sm, n, size, quantised):
    """chunk_attend's rows with a slack that counts only what a row sees and weighs.

    With t_j the largest value of key j's block (size: 16, few rows 32) and u = 2^-11:
    weights as there; a value entry is off by 4 u t_j at most where it is a rounded
    minimum (t_j) plus a rounded scale times a code (2 t_j), rounded (t_j), and by
    2^-18 t_j where it is exact (half a subnormal step, 2^-25, beside a largest entry
    of 2^-7 or more); a weight below 2^-14 of the outputs' scale 2^R is off by 2^-25
    of that.  2^R is at most twice max_j p_j 2^(e_j), and the block's power of two
    2^(e_j) puts its largest entry into [2^(c-1), 2^c) for one c, all entries below
    2^c: 2^-25 x 2 x 2 max_j(p_j t_j) = 2^-23 max_j(p_j t_j) for each key.
    """
    top = block_tops(vh, n, size)
    want, slack = np.zeros(q.shape), np.zeros(q.shape)
    u = 2.0**-11
    entry = 4 * u if quantised else 2.0**-18
    for i in range(q.shape[0]):
        k, v, t = kh[: last[i] + 1], vh[: last[i] + 1], top[: last[i] + 1]
        s = sm * (k @ q[i])
        e = np.exp(s - s.max())
        p = e / e.sum()
        want[i] = p @ v
        dj = (u + q.shape[1] * 2.0**-23) * abs(sm) * (np.abs(k) @ np.abs(q[i]))
        w = p * (dj + p @ dj + u + 2.0**-16)
        slack[i] = 1.05 * (w @ np.abs(v) + entry * (p @ t) + len(p) * 2.0**-23 * (p * t).max()) + 2.0**-8 * np.abs(want[i])
    return want, slack


def far_case(m, kind, d, T, start, current, change, seed=0, sm=0.5, B=1, heads=2, rows=None):
    n = start if current else start + T
    k, v = (seeded_bf16((B, start + T, 1, d), seed + i) for i in range(2))
    q = seeded_bf16((B, T, heads, d), seed + 2, 0.3)
    change(q, k, v)
    kv, table = cell_for(m, kind, B, 1, d, max(n, 1), heads, seed)
    m.loopkv_rope_append(kv, 0, 0, None, None, k[:, :n], v[:, :n], table, ints([0] * B))
    cur = dict(k_cur=k[:, n:], v_cur=v[:, n:]) if current else {}
    out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([start] * B), sm_scale=sm, **cur)
    rows = np.arange(T) if rows is None else np.asarray(rows)
    quantised = kind != "bf16"
    size = 32 if quantised and T * heads <= 16 else 16
    for b in range(B):
        kh, vh = CO.stored_values(kind, host(k[b, :n, 0]), host(v[b, :n, 0]))
        kh, vh = np.vstack([kh, host(k[b, n:, 0])]).astype(np.float64), np.vstack([vh, host(v[b, n:, 0])]).astype(np.float64)
        for h in range(heads):
            want, slack = attend_seen(host(q[b, rows, h]).astype(np.float64), kh, vh, start + rows, sm, n, size, quantised)
            off = np.abs(host(out[b, rows, h]) - want)
            assert np.all(off <= slack), (b, h, float((off / slack).max()), int((off / slack).max(1).argmax()))


@pytest.mark.parametrize("kind,current", [("q4", False), ("q2", False), ("bf16", False), ("q4", True), ("bf16", True)])
@pytest.mark.parametrize("big", [2.0**14, 2.0**20, 2.0**26, 2.0**40, 2.0**90])
@pytest.mark.parametrize("T,start,first", [(150, 0, 16), (150, 0, 64), (140, 0, 128), (8, 28, 32), (300, 20, 160)])
def test_values_that_a_row_does_not_see(m, kind, current, big, T, start, first):
    """Later tokens' values are far larger than those that the early rows see."""
    if current and T < 100:
        pytest.skip("the chunk's few rows are one block")
    at = start + (first - start + 15) // 16 * 16 if current else first     # where a block begins

    def change(q, k, v):
        v[:, at:] *= big

    far_case(m, kind, 64, T, start, current, change)


@pytest.mark.parametrize("kind,current", [("q4", False), ("q2", False), ("bf16", False), ("q4", True)])
@pytest.mark.parametrize("big,down", [(2.0**16, 30), (2.0**24, 40), (2.0**40, 70), (2.0**60, 80), (2.0**40, 20), (2.0**100, 150)])
@pytest.mark.parametrize("T,start", [(7, 500), (150, 500), (150, 1900)])
def test_large_values_of_little_weight(m, kind, current, big, down, T, start):
    """Some groups have values far larger, and logits far smaller (by 2^-down of the
    weight): what they add is as little or as much as it is."""
    def change(q, k, v):
        k[..., 0] = 0
        q[..., 0] = 1.0
        for lo in (0, 96, 288):
            k[:, lo: lo + 32, :, 0] = -2 * down * np.log(2.0)      # sm = 0.5
            v[:, lo: lo + 32] *= big
        k[:, 416: 448, :, 0] = 20.0                                 # late in the context the maximum moves up
    far_case(m, kind, 64, T, start, current, change, seed=4, rows=range(0, T, max(1, T // 12)))


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("current", [False, True])
@pytest.mark.parametrize("T,start", [(5, 1500), (5, 40), (140, 1500), (300, 40)])
@pytest.mark.parametrize("v_scale", [2.0**118, 2.0**125, 2.0**-110])
def test_values_at_the_ends_of_the_range(m, kind, current, T, start, v_scale):
    """Averages of values near the largest number, and of very small ones."""
    def change(q, k, v):
        v.copy_((v.float().clamp(-3, 3).abs() if v_scale > 2.0**120 else v.float()).mul(v_scale).bfloat16())
    far_case(m, kind, 64, T, start, current, change, seed=8, rows=range(0, T, max(1, T // 9)))


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("current", [False, True])
@pytest.mark.parametrize("T,start", [(5, 100), (140, 100)])
@pytest.mark.parametrize("k_pow,q_pow,s_pow", [(121, 0, -121), (121, -121, 0), (121, -60, -61), (-90, 100, -10), (-90, 0, 90),
                                               (90, 36, -126), (-60, -60, 120), (60, -100, 40)])
def test_keys_queries_and_scale_far_from_one(m, kind, current, T, start, k_pow, q_pow, s_pow):
    """Logits of ordinary size out of keys, queries and a scale that are not."""
    def change(q, k, v):
        k.mul_(2.0**k_pow)
        q.mul_(2.0**q_pow)
    far_case(m, kind, 64, T, start, current, change, seed=12, sm=0.5 * 2.0**s_pow, rows=range(0, T, max(1, T // 9)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [1, 2])
def test_all_columns_weigh_alike(m, d, heads):
    """Keys of one logit have one weight, whether its exponential is the unit's or
    the polynomial's (columns 6 and 7 of eight), over many fractions of the exponent.

    Values 1 in six columns and -3 in two cancel: with w the keys' weight beside one
    of weight 1, 48 n (w' - w'') / (1 + 64 n w) remains of n x 64 keys, where w' and w''
    differ by 7.6e-5 (the cubic) + 2 x 2^-11 (both rounded to fp16) + 2^-20 (the unit,
    sums) of w; then the output's rounding.
    """
    T, n = 150, 3
    k = torch.zeros(1, 64 * n + 8, 1, d, device="cuda")
    v = torch.zeros_like(k)
    k[:, 1:8, :, 0] = -60000.0                  # no weight; key 0, of logit 0, comes first and is the reference
    k[:, 8:, :, 0] = -1
    v[:, 8:] = torch.where(torch.arange(64 * n, device="cuda") % 8 < 6, 1.0, -3.0)[None, :, None, None]
    k, v = k.bfloat16(), v.bfloat16()
    q = torch.zeros(1, T, heads, d, device="cuda")
    q[0, :, :, 0] = torch.linspace(0.01, 4, T, device="cuda")[:, None] + 0.013 * torch.arange(heads, device="cuda")
    q = q.bfloat16()
    cur = torch.zeros(1, T, 1, d, dtype=torch.bfloat16, device="cuda")
    kc = cur.clone()
    kc[..., 0] = -60000.0                       # the chunk's own rows: no weight
    kv, table = cell_for(m, "bf16", 1, 1, d, 64 * n + 8, heads)
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0]))
    out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([64 * n + 8]), sm_scale=1.0, k_cur=kc, v_cur=cur)
    w = np.exp(-host(q[0, :, :, 0]).astype(np.float64))
    bound = 48 * n * w * (7.6e-5 + 2 * 2.0**-11 + 2.0**-20) / (1 + 64 * n * w * (1 - 2.0**-9)) * (1 + 2.0**-8)
    off = np.abs(host(out[0])).max(-1)
    assert np.all(off <= bound), float((off / bound).max())
    assert off.max() > 0                        # the two do differ
