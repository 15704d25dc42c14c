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


def same_bytes(a, b, lens):
    assert torch.equal(a.arenas[0], b.arenas[0])
    if a.residuals[0] is not None:
        for i, n in enumerate(lens):
            assert torch.equal(bits(a.residuals[0][i, :, : n % 32]), bits(b.residuals[0][i, :, : n % 32]))


def odd_entries(x, seed):
    """Single entries, whole 32-channel groups and whole 32-token columns of x [B, T, heads, D] that are not finite."""
    g = torch.Generator().manual_seed(seed)
    B, T, H, D = x.shape
    for value in (NAN, INF, -INF, NAN, INF, 3.3e38, -3.3e38):
        for _ in range(6):
            b, t, h, c = (int(torch.randint(0, n, (1,), generator=g)) for n in x.shape)
            x[b, t, h, c] = value
        x[b, (t + 5) % T, h, c // 32 * 32: c // 32 * 32 + 32] = value
        x[b, : T // 32 * 32, h, (c + 1) % D] = value
    bits(x)[0, 1, 0, 3], bits(x)[0, 2, 0, 4] = -1, 0x7F81        # NaN of other bits
    return x


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("turned", [False, True])
def test_append_of_what_is_not_finite(m, kind, d, turned):
    """The bytes of norm_rope and quantize_append, NaN and infinities included."""
    B, hkv, steps = 3, 2, [[70, 64, 5], [1, 31, 27], [33, 1, 64]]
    r = rotary_for(m, d, d // 2, False, True)[0] if turned else None
    got, table = cell_for(m, kind, B, hkv, d, 200)
    want, _ = cell_for(m, kind, B, hkv, d, 200)
    have = [0] * B
    for step, lens in enumerate(steps):
        T = max(lens)
        k, v = (odd_entries(seeded_bf16((B, T, hkv, d), 40 + 2 * step + i), 7 + 2 * step + i) for i in range(2))
        start = ints(have)
        m.loopkv_rope_append(got, 0, 0, r, None, k, v, table, start, ints(lens))
        k_in = m.loopkv_norm_rope(r or m.Rotary(), None, k, start, ints(lens))[1]
        for b, n in enumerate(lens):
            one = ints([have[b] if i == b else -1 for i in range(B)])
            m.loopkv_quantize_append(want, 0, 0, k_in[:, :n].contiguous(), v[:, :n].contiguous(), table, one)
        have = [a + n for a, n in zip(have, lens)]
        same_bytes(got, want, have)


# ---------------------------------------------------------------- attention


def attend_any(q, kh, vh, last, sm):
    """chunk_attend's rows and slack where keys and values need not be finite: a row
    with a NaN or +inf logit (or -inf alone) is NaN, a logit of -inf has no weight, and
    a value that is not finite goes into its channel of every row that sees it."""
    rows, d = q.shape
    want, slack = np.full((rows, d), np.nan), np.zeros((rows, d))
    clean = np.where(np.isfinite(vh), vh, 0.0)
    for i in range(rows):
        n = last[i] + 1
        with np.errstate(all="ignore"):
            s = sm * (kh[:n] @ q[i])
        if np.isnan(s).any() or s.max() == np.inf or s.max() == -np.inf:
            continue
        keep = np.isfinite(s)
        w, e = CO.chunk_attend(q[i: i + 1], kh[:n][keep], clean[:n][keep], [int(keep.sum()) - 1], sm)
        with np.errstate(all="ignore"):
            odd = np.where(np.isfinite(vh[:n]), 0.0, vh[:n])[keep].sum(0)
        want[i], slack[i] = w[0] + odd, e[0]
    return want, slack


def check(out, want, slack, what):
    got, fine = host(out).astype(np.float64), np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    odd = ~fine & ~np.isnan(want)
    assert np.array_equal(got[odd], want[odd]), what
    assert np.all(np.abs(got - np.where(fine, want, 0))[fine] <= slack[fine]), what


def run_case(m, kind, d, T, start, current, spoil, seed=0, sm=0.6, B=8, heads=2, hkv=1):
    """A chunk behind `start` tokens in each of B sequences; spoil(b, q, k, v, stored) puts
    into sequence b what is not finite, k and v over stored and current tokens."""
    n = start if current else start + T
    k, v = (seeded_bf16((B, start + T, hkv, d), seed + i) for i in range(2))
    q = seeded_bf16((B, T, heads, d), seed + 2, 0.3)
    for b in range(B):
        spoil(b, q[b], k[b], v[b], n)
    kv, table = cell_for(m, kind, B, hkv, d, max(n, 1), heads, seed)
    m.loopkv_rope_append(kv, 0, 0, None, None, k[:, :n], v[:, :n], table, ints([0] * B))
    cur = dict(k_cur=k[:, n:], v_cur=v[:, n:]) if current else {}
    err = ints([0])
    out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([start] * B), sm_scale=sm, err_flag=err, **cur)
    assert int(err) == 0
    return k, v, q, out


def exact_rows(kind, k, v, n, h):
    """Keys and values of KV head h as they are stood for, all of them finite before."""
    kh, vh = CO.stored_values(kind, host(k[:n, h]), host(v[:n, h]))
    return np.vstack([kh, host(k[n:, h]).astype(np.float64)]), np.vstack([vh, host(v[n:, h]).astype(np.float64)])


PLACES = [("bf16", 64, 12, 10, False), ("bf16", 128, 140, 10, False), ("q4", 128, 12, 10, False), ("q4", 64, 140, 10, False),
          ("q2", 128, 140, 10, False), ("q4", 128, 12, 40, True), ("q2", 64, 12, 33, True), ("q4", 128, 140, 40, True),
          ("bf16", 64, 140, 40, True), ("bf16", 128, 12, 3, True)]


@pytest.mark.parametrize("kind,d,T,start,current", PLACES)
def test_a_nan_key_shows_whatever_its_place(m, kind, d, T, start, current):
    """Every row that sees a key with a NaN is NaN, at each place of eight."""
    at = [start + (3 if T < 100 else 121) + b for b in range(8)]     # in the open group of 32

    def spoil(b, q, k, v, n):
        k[at[b], 0, 5] = NAN

    _, _, _, out = run_case(m, kind, d, T, start, current, spoil)
    for b in range(8):
        assert torch.isnan(out[b, at[b] - start:]).all() and not torch.isnan(out[b, : at[b] - start]).any()


@pytest.mark.parametrize("kind,d,T,start,current", PLACES)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_keys_that_are_not_finite(m, kind, d, T, start, current, value):
    """An exact key with one such entry, at each place of eight: rows before it
    are as without it, rows that see it are NaN, or have no weight for it where
    its logit is -inf."""
    B = 8
    at = [start + (3 if T < 100 else 121) + b for b in range(B)]     # in the open group of 32

    def spoil(b, q, k, v, n):
        k[at[b], 0, 5] = value

    k, v, q, out = run_case(m, kind, d, T, start, current, spoil, B=B)
    n = start if current else start + T
    for b in range(B):
        clean = k[b].clone()
        clean[at[b], 0, 5] = 0
        kh, vh = exact_rows(kind, clean, v[b], n, 0)
        kh[at[b], 5] = value
        for h in range(2):
            want, slack = attend_any(host(q[b, :, h]).astype(np.float64), kh, vh, start + np.arange(T), 0.6)
            check(out[b, :, h], want, slack, (b, h))


@pytest.mark.parametrize("kind", ["q4", "bf16"])
@pytest.mark.parametrize("T,start", [(5, 0), (150, 0), (5, 1500), (150, 1500)])
def test_queries_that_are_not_finite(m, kind, T, start):
    """One head's row with a NaN, one with an infinity: those rows are NaN, however
    the context is split, and no others change."""
    def spoil(b, q, k, v, n):
        q[1, 0, 7], q[3, 1, 0], q[T - 1, 1, 3] = NAN, INF, -INF
        k[:, 0, 3] = k[:, 0, 3].abs() + 0.1      # so that all of that row's logits are -inf

    k, v, q, out = run_case(m, kind, 128, T, start, False, spoil, B=2)
    for b in range(2):
        kh, vh = exact_rows(kind, k[b], v[b], start + T, 0)
        for h in range(2):
            want, slack = attend_any(host(q[b, :, h]).astype(np.float64), kh, vh, start + np.arange(T), 0.6)
            bad = {0: {1}, 1: {3, T - 1}}[h]
            assert {i for i in range(T) if np.isnan(want[i]).any()} == bad
            check(out[b, :, h], want, slack, (b, h))


@pytest.mark.parametrize("kind,d,T,start,current", PLACES)
def test_values_that_are_not_finite(m, kind, d, T, start, current):
    """A value's infinity or NaN reaches its channel of the rows that see it, and
    nothing else; two infinities of both signs meet as NaN."""
    B, n = 8, start if current else start + T
    odd = {}

    def spoil(b, q, k, v, n):
        j = start + (2 if T < 100 else 118) + b
        odd[b] = [(j, 1, [INF, -INF, NAN, INF][b % 4]), (j + 1, 40, -INF), (j + 2, 40, INF), (min(b, start - 1), 2, NAN)]
        for t, c, x in odd[b]:
            if t < n and kind != "bf16":           # a quantised group of 32 channels goes as a whole
                v[t, 0, c // 32 * 32: c // 32 * 32 + 32] = x
            else:
                v[t, 0, c] = x

    k, v, q, out = run_case(m, kind, d, T, start, current, spoil, seed=5, B=B)
    for b in range(B):
        clean = torch.where(torch.isfinite(v[b]), v[b], torch.zeros_like(v[b]))
        kh, vh = exact_rows(kind, k[b], clean, n, 0)
        for t, c, x in odd[b]:
            if t < n and kind != "bf16":
                vh[t, c // 32 * 32: c // 32 * 32 + 32] = np.nan     # inf times the code 0
            else:
                vh[t, c] = x
        for h in range(2):
            want, slack = attend_any(host(q[b, :, h]).astype(np.float64), kh, vh, start + np.arange(T), 0.6)
            check(out[b, :, h], want, slack, (b, h))


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("T", [9, 200])
def test_values_that_are_not_finite_in_a_split_context(m, kind, T):
    """The same with the context split over CTAs, and with whole rows of values."""
    start, d = 1400, 128
    places = [100, 101, 1403, start + T - 3]

    def spoil(b, q, k, v, n):
        v[places[0], 0, 32:64], v[places[1], 0, 64:96] = INF, NAN
        v[places[2], 0], v[places[3], 0] = NAN, -INF

    k, v, q, out = run_case(m, kind, d, T, start, False, spoil, seed=9, B=2)
    for b in range(2):
        clean = torch.where(torch.isfinite(v[b]), v[b], torch.zeros_like(v[b]))
        kh, vh = exact_rows(kind, k[b], clean, start + T, 0)
        raw = host(v[b, :, 0]).astype(np.float64)
        vh = np.where(np.isfinite(raw), vh, raw if kind == "bf16" else np.nan)
        for h in range(2):
            want, slack = attend_any(host(q[b, :, h]).astype(np.float64), kh, vh, start + np.arange(T), 0.6)
            check(out[b, :, h], want, slack, (b, h))


@pytest.mark.parametrize("kind", ["q4", "q2"])
@pytest.mark.parametrize("T,start", [(8, 88), (140, 0)])
def test_a_quantised_key_group_that_is_not_finite(m, kind, T, start):
    """An infinite key makes its channel's scale infinite: the whole group of 32
    tokens has no logits, and rows before it are as they were."""
    def spoil(b, q, k, v, n):
        k[70, 0, 9] = INF

    k, v, q, out = run_case(m, kind, 128, T, start, False, spoil, seed=3, B=2)
    for b in range(2):
        clean = k[b].clone()
        clean[70, 0, 9] = 0
        kh, vh = exact_rows(kind, clean, v[b], start + T, 0)
        kh[64:96, 9] = np.nan
        for h in range(2):
            want, slack = attend_any(host(q[b, :, h]).astype(np.float64), kh, vh, start + np.arange(T), 0.6)
            check(out[b, :, h], want, slack, (b, h))


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("T", [6, 150])
@pytest.mark.parametrize("every", [1, 9000])
def test_many_values_that_are_not_finite(m, kind, T, every):
    """Infinities in one channel group of all tokens, or far apart, in a long context."""
    n, d = 18_100, 64
    kv, table = cell_for(m, kind, 1, 1, d, n)
    k, v, q = (seeded_bf16((1, n, 1, d), i) for i in range(3))
    v[:, ::every, :, 32:] = INF
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0]))
    q = q[:, :T].contiguous()
    out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([n - T]), sm_scale=0.1)
    v[:, ::every, :, 32:] = 0
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0]))
    want = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([n - T]), sm_scale=0.1)
    assert torch.equal(out[..., :32], want[..., :32])
    assert torch.isnan(out[..., 32:]).all() if kind != "bf16" else torch.isposinf(out[..., 32:]).all()


@pytest.mark.parametrize("eps", [1e75, 1e300])
def test_norms_under_a_huge_eps(m, eps):
    """Every row's norm is as small as that of a row of infinities; rows that are not there are not read."""
    w = seeded_bf16((64,), 3, 0.2) + 1
    r = m.Rotary(m.rope_table(50, 64), q_weight=w, k_weight=w, eps=eps)
    x = seeded_bf16((2, 7, 3, 64), 1, 1e37)
    lens = [7, 2]
    out = m.loopkv_norm_rope(r, x[:, :, :1], x[:, :, 1:], ints([3, 40]), ints(lens))
    kv, table = cell_for(m, "q4", 2, 2, 64, 64, 2)
    m.loopkv_rope_append(kv, 0, 0, r, None, x[:, :, 1:], x[:, :, 1:], table, ints([3, 40]), ints(lens))
    with np.errstate(all="ignore"):
        for b, (s, n) in enumerate([(3, 7), (40, 2)]):
            for o, i in zip(out, (slice(0, 1), slice(1, 3))):
                want = CO.norm_rope(host(x[b, :n, i]), s + np.arange(n), host(r.table), weight=host(w), eps=eps)
                assert np.array_equal(host(o[b, :n]), want) and not o[b, n:].any()
                if i.start:
                    got = kv.residuals[0][b, :, s % 32: s % 32 + n].transpose(0, 1)
                    assert np.array_equal(host(got), want)


@pytest.mark.parametrize("kind,T,start,current", [("q4", 150, 1500, True), ("bf16", 150, 1500, False), ("bf16", 300, 20, True),
                                                  ("q4", 8, 1500, False), ("q2", 8, 1500, False), ("q4", 3, 1503, False)])
def test_a_nan_stays_where_nothing_follows(m, kind, T, start, current):
    """A row that sees a NaN logit and after it only keys that it masks is NaN,
    however the context is split over CTAs and warps."""
    B = 3
    few = T < 16
    last = (start + T - 1) // 32                                     # the last group, masked for the chunk's first rows
    at = [32 * (last - back) + 1 if few else start + 5 + 40 * b for b, back in enumerate((3, 6, 12))]

    def spoil(b, q, k, v, n):
        k[at[b], 0, 9] = INF if few else NAN                          # a full group of a quantised cell goes as a whole

    _, _, _, out = run_case(m, kind, 64, T, start, current, spoil, B=B)
    for b in range(B):
        first = 0 if few else at[b] - start
        assert torch.isnan(out[b, first:]).all() and not torch.isnan(out[b, :first]).any()


def split_case(m, kind, start, T, heads, spoil):
    """One sequence's chunk of current rows in a cell whose capacity is far larger: its
    few keys are met by some warps of some CTAs, the others see none."""
    k, v, q = seeded_bf16((1, start + T, 1, 64), 1), seeded_bf16((1, start + T, 1, 64), 2), seeded_bf16((1, T, heads, 64), 3, 0.3)
    spoil(k[0, :, 0], v[0, :, 0])
    kv, table = cell_for(m, kind, 1, 1, 64, 4000, heads)
    m.loopkv_rope_append(kv, 0, 0, None, None, k[:, :start], v[:, :start], table, ints([0]))
    return m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([start]), k_cur=k[:, start:], v_cur=v[:, start:])


@pytest.mark.parametrize("kind,start", [("q2", 30), ("q4", 30), ("q2", 62), ("q4", 100), ("q2", 333), ("bf16", 400)])
@pytest.mark.parametrize("T,heads", [(1, 8), (2, 8), (60, 2)])
def test_a_nan_key_in_one_part_of_a_split_context(m, kind, start, T, heads):
    """A part whose rows have no logit but a NaN still counts in the join."""
    def spoil(k, v):
        k[start - 1, 5] = NAN                                         # in the open group

    assert torch.isnan(split_case(m, kind, start, T, heads, spoil)).all()


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("T,heads", [(1, 8), (2, 8), (60, 2)])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_infinite_values_beside_far_larger_ones(m, kind, T, heads, value):
    """A part with nothing but infinite values joins parts of values of 2^30: its
    share of them is not 0 times infinity."""
    def spoil(k, v):
        v[:40] *= 2.0**30
        v[40] = value                                                 # the first current row

    out = split_case(m, kind, 40, T, heads, spoil)
    assert torch.isnan(out).all() if value != value else (out == value).all()
