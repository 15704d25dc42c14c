"""NaN and infinities on the prompt side: a row shows those that it sees, and
no others, wherever they stand in a block, a group or a tile."""

import numpy as np
import pytest
import torch

from loopkv_testlib import seeded_bf16
from oracle import chunk_oracle as CO
from test_gpu_chunk import cell_for, fused_rows, host, ints, rotary_for

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def m():
    import mixed_precision_kv_loopkv_b200 as pkg
    return pkg


def bits(t):
    return t.view(torch.int16)


def odd_rows(x, first=0):
    """Some rows of x [B, T, heads, D] get a NaN, infinities, or numbers whose squares are beyond fp32."""
    flat = x.view(-1, x.shape[-1])
    n = flat.shape[0]
    for i, (channel, value) in enumerate([(1, NAN), (5, INF), (x.shape[-1] - 1, -INF), (0, 3e38), (9, -1e30), (17, NAN)]):
        flat[(first + 7 * i + i // 2) % n, channel] = value
    flat[(first + 50) % n, 3:6] = INF
    flat[(first + 51) % n] = 3e38                 # a finite row whose squares add up to more than 2^254
    flat[(first + 52) % n] = NAN
    return x


@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (128, 64, True), (64, 32, False), (64, 0, False)])
@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (2, 1)])
def test_norms_of_rows_that_are_not_finite(m, d, rot, interleaved, heads, kv_heads):
    """The mean of a row's squares is NaN or infinite where one of its entries is:
    the row is NaN, or zeros with a NaN."""
    B, T = 2, 17
    r, qa, ka = rotary_for(m, d, rot, interleaved, True)
    q, k = odd_rows(seeded_bf16((B, T, heads, d), 1)), odd_rows(seeded_bf16((B, T, kv_heads, d), 2), 3)
    start = [4, 900]
    q_out, k_out = m.loopkv_norm_rope(r, q, k, ints(start))
    assert torch.isnan(q_out).any() and torch.isnan(k_out).any()
    kv, table = cell_for(m, "bf16", B, kv_heads, d, 1000, heads)
    q_app = m.loopkv_rope_append(kv, 0, 0, r, q, k, k, table, ints(start))
    k_app = m.loopkv_read_tokens(kv, 0, 0, table, ints([s + T for s in start]), ints(start), T)[0]
    with np.errstate(all="ignore"):
        for x, outs, a in ((q, (q_out, q_app), qa), (k, (k_out, k_app), ka)):
            for b in range(B):
                want = CO.norm_rope(host(x[b]), start[b] + np.arange(T), **a)
                for o in outs:
                    assert np.array_equal(host(o[b]), want, equal_nan=True)
