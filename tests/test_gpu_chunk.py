"""GPU parity of the prompt side: norms and rotation, rotated append, reading
back, and chunk attention, each against the plain oracle."""

import numpy as np
import pytest
import torch

from loopkv_testlib import seeded_bf16
from oracle import chunk_oracle as CO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mixed_precision_kv_loopkv_b200 as pkg
    return pkg


def ints(xs):
    return torch.tensor(list(xs), dtype=torch.int32, device="cuda")


def host(t):
    return t.float().cpu().numpy()


def rotary_for(m, d, rot, interleaved, norm, positions=1200, seed=3):
    """(Rotary, arguments of the oracle's norm_rope for q and for k)."""
    table = None if rot == 0 else torch.from_numpy(CO.rope_angles(positions, rot)).cuda()
    qw, kw = ((seeded_bf16((d,), seed + i, 0.2) + 1) if norm else None for i in (0, 1))
    r = m.Rotary(table, interleaved=interleaved, q_weight=qw, k_weight=kw, eps=1e-5)
    t = None if table is None else host(table)
    args = [dict(table=t, interleaved=interleaved, weight=None if w is None else host(w), eps=1e-5) for w in (qw, kw)]
    return r, args[0], args[1]


def fused_rows(batch, tokens, heads, kv_heads, d, seed):
    """q, k, v as views of one projection's output."""
    x = seeded_bf16((batch, tokens, (heads + 2 * kv_heads) * d), seed)
    return tuple(y.unflatten(-1, (-1, d)) for y in x.split([heads * d, kv_heads * d, kv_heads * d], -1))


ROTATIONS = [(128, 128, False, True), (128, 64, True, True), (128, 128, True, False), (64, 64, False, True),
             (64, 16, False, False), (64, 48, True, True), (128, 96, False, True), (64, 0, False, True)]


@pytest.mark.parametrize("d,rot,interleaved,norm", ROTATIONS)
@pytest.mark.parametrize("heads,kv_heads,tokens", [(4, 2, 1), (5, 5, 37), (8, 1, 130)])
def test_norm_rope_bits(m, d, rot, interleaved, norm, heads, kv_heads, tokens):
    B = 3
    r, qa, ka = rotary_for(m, d, rot, interleaved, norm)
    q, k, _ = fused_rows(B, tokens, heads, kv_heads, d, seed=11)
    q[0, 0, 0] = 0                                   # a row of zeros has a norm of its eps
    start, lens = [0, 1000, -1], [tokens, max(1, tokens // 2), tokens]
    err = ints([0])
    q_out = torch.full((B, tokens, heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((B, tokens, kv_heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    m.loopkv_norm_rope(r, q, k, ints(start), ints(lens), q_out, k_out, err_flag=err)
    for x, o, a in ((q, q_out, qa), (k, k_out, ka)):
        for b in range(B):
            n = lens[b] if start[b] >= 0 else 0
            want = CO.norm_rope(host(x[b, :n]), start[b] + np.arange(n), **a)
            assert np.array_equal(host(o[b, :n]), want)
            assert (o[b, n:] == 7).all()             # rows behind are left as they were
    assert int(err) == 0


def test_norm_rope_in_place_and_alone(m):
    r, qa, ka = rotary_for(m, 64, 64, False, True)
    q, k = seeded_bf16((2, 9, 3, 64), 1), seeded_bf16((2, 9, 2, 64), 2)
    want_q = [CO.norm_rope(host(q[b]), 5 + b + np.arange(9), **qa) for b in range(2)]
    want_k = [CO.norm_rope(host(k[b]), 5 + b + np.arange(9), **ka) for b in range(2)]
    got_q, none = m.loopkv_norm_rope(r, q, None, ints([5, 6]))
    assert none is None
    none, got_k = m.loopkv_norm_rope(r, None, k, ints([5, 6]))
    assert none is None
    m.loopkv_norm_rope(r, q, k, ints([5, 6]), q_out=q, k_out=k)
    for b in range(2):
        for got in (got_q, q):
            assert np.array_equal(host(got[b]), want_q[b])
        for got in (got_k, k):
            assert np.array_equal(host(got[b]), want_k[b])


def test_norm_rope_faults(m):
    r, _, _ = rotary_for(m, 64, 64, False, False, positions=20)
    q = seeded_bf16((4, 6, 1, 64), 1)
    out = torch.full_like(q, 3.0)
    err = ints([0])
    # beyond the table; more rows than there are; fewer than none; nothing to do far out
    m.loopkv_norm_rope(r, q, None, ints([15, 0, 0, 2**31 - 1]), ints([6, 7, -1, 0]), q_out=out, err_flag=err)
    assert int(err) == m.LOOPKV_DEVERR_SEQ_LEN and (out == 3).all()


def cell_for(m, kind, B, hkv, d, capacity, heads=None, seed=5):
    rng = np.random.default_rng(seed)
    mb = -(-capacity // 16)
    pool = B * mb + 7
    ids = rng.permutation(pool)[: B * mb].reshape(B, mb).astype(np.int32)
    kv = m.KVCells([kind], 1, 1, heads or hkv, d, pool, B, mb, num_kv_heads=hkv)
    return kv, torch.from_numpy(ids).cuda()


def same_cell(a, b, lens):
    assert torch.equal(a.arenas[0], b.arenas[0])
    if a.residuals[0] is not None:
        for i, n in enumerate(lens):
            assert torch.equal(a.residuals[0][i, :, : n % 32], b.residuals[0][i, :, : n % 32])


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("d,rot,interleaved,norm", [(128, 128, False, True), (64, 32, True, True), (128, 64, True, False)])
def test_rope_append_stores_what_the_two_calls_store(m, kind, d, rot, interleaved, norm):
    """Chunks of every kind of length and place, ragged and with skipped
    sequences: byte for byte what norm_rope and quantize_append store."""
    B, hkv, heads, cap = 5, 3, 6, 400
    r, qa, _ = rotary_for(m, d, rot, interleaved, norm)
    got, table = cell_for(m, kind, B, hkv, d, cap, heads)
    want, _ = cell_for(m, kind, B, hkv, d, cap, heads)
    have = [0] * B
    err = ints([0])
    for step, lens in enumerate([[1, 31, 32, 33, 70], [1, 1, 0, 40, 0], [30, 5, 64, 23, 1], [100, 27, 1, 97, 26],
                                 [1, 1, 1, 1, 1], [127, 96, 3, 64, 95]]):
        T = max(lens) + step % 2
        skip = step % B
        q, k, v = fused_rows(B, T, heads, hkv, d, seed=100 + step)
        start = [-1 if b == skip and step else have[b] for b in range(B)]
        q_out = torch.full((B, T, heads, d), 5.0, dtype=torch.bfloat16, device="cuda")
        m.loopkv_rope_append(got, 0, 0, r, q, k, v, table, ints(start), ints(lens), q_out, err_flag=err)
        k_rot = m.loopkv_norm_rope(r, None, k, ints(start), ints(lens))[1]
        for n in sorted(set(lens) - {0}):
            one = [start[b] if lens[b] == n else -1 for b in range(B)]
            m.loopkv_quantize_append(want, 0, 0, k_rot[:, :n].contiguous(), v[:, :n].contiguous(), table, ints(one))
        for b in range(B):
            n = lens[b] if start[b] >= 0 else 0
            assert np.array_equal(host(q_out[b, :n]), CO.norm_rope(host(q[b, :n]), start[b] + np.arange(n), **qa))
            assert (q_out[b, n:] == 5).all()
            have[b] += n
        same_cell(got, want, have)
    assert int(err) == 0


@pytest.mark.parametrize("kind", ["q4", "q2"])
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 300.0, 1e30])
def test_rope_append_codes_at_extreme_scales(m, kind, scale):
    """The codes come from a product with 1/s where that decides; the bytes are
    those of the division at scales far from one too, and on ties."""
    B, hkv, d, T = 2, 2, 64, 96
    k, v = (seeded_bf16((B, T, hkv, d), 20 + i, scale) for i in range(2))
    k[0, :32] = (torch.arange(32, device="cuda") % 4 * 0.5 * 2.0**-3)[:, None, None]   # halves of a step
    v[1, :, :, 32:] = (torch.arange(32, device="cuda") * 0.5).bfloat16()
    v[1, 5] = 0.75                                                                       # a group of one value
    got, table = cell_for(m, kind, B, hkv, d, T)
    want, _ = cell_for(m, kind, B, hkv, d, T)
    m.loopkv_rope_append(got, 0, 0, None, None, k, v, table, ints([0, 0]))
    m.loopkv_quantize_append(want, 0, 0, k, v, table, ints([0, 0]))
    same_cell(got, want, [T, T])


def test_rope_append_faults(m):
    got, table = cell_for(m, "q4", 3, 2, 64, 64)
    k, v = seeded_bf16((3, 40, 2, 64), 1), seeded_bf16((3, 40, 2, 64), 2)
    err = ints([0])
    m.loopkv_rope_append(got, 0, 0, None, None, k, v, table, ints([30, 0, 64]), ints([40, 41, 0]), err_flag=err)
    assert int(err) == m.LOOPKV_DEVERR_SEQ_LEN and not got.arenas[0].any() and not got.residuals[0].any()
    err.zero_()
    table[0, 0], table[2, 1] = -1, 10_000
    m.loopkv_rope_append(got, 0, 0, None, None, k, v, table, ints([0, 0, 0]), err_flag=err)
    assert int(err) == m.LOOPKV_DEVERR_BLOCK_ID
    good, _ = cell_for(m, "q4", 3, 2, 64, 64)
    m.loopkv_rope_append(good, 0, 0, None, None, k, v, cell_for(m, "q4", 3, 2, 64, 64)[1], ints([0, 0, 0]))
    touched = got.arena_view(0).flatten(1).any(1)
    for b in range(3):
        for j in range(3):
            blk = int(table[b, j])
            if 0 <= blk < got.num_blocks:
                assert torch.equal(got.arena_view(0)[blk], good.arena_view(0)[blk])
                touched[blk] = False
    assert not touched.any()            # and nothing else was written


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_read_tokens(m, kind, d):
    B, hkv, cap = 4, 3, 200
    kv, table = cell_for(m, kind, B, hkv, d, cap)
    k, v = seeded_bf16((B, cap, hkv, d), 1, 3.0), seeded_bf16((B, cap, hkv, d), 2)
    lens = [200, 77, 1, 32]
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0] * B), ints(lens))
    stands = [[CO.stored_values(kind, host(k[b, :lens[b], h]), host(v[b, :lens[b], h])) for h in range(hkv)] for b in range(B)]
    for start, count in ([0, 0, 0, 0], 200), ([3, 64, 0, 31], 45), ([199, 76, -1, 32], 1), ([150, 77, 5, 2**31 - 1], 64):
        outs = [torch.full((B, count, hkv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        err = ints([0])
        m.loopkv_read_tokens(kv, 0, 0, table, ints(lens), ints(start), count, *outs, err_flag=err)
        assert int(err) == 0
        for b in range(B):
            n = max(0, min(count, lens[b] - start[b])) if start[b] >= 0 else 0
            for h in range(hkv):
                for o, w in zip(outs, stands[b][h]):
                    want = torch.from_numpy(w[start[b]: start[b] + n].astype(np.float32)).bfloat16()
                    assert torch.equal(o[b, :n, h].cpu(), want)
                    assert (o[b, n:] == 9).all()
    new = m.loopkv_read_tokens(kv, 0, 0, table, ints(lens), ints([0] * B), 33)
    assert not new[0][2, 1:].any() and new[1][0].any()


def test_read_tokens_faults(m):
    kv, table = cell_for(m, "q4", 2, 1, 64, 64)
    k, v = seeded_bf16((2, 64, 1, 64), 1), seeded_bf16((2, 64, 1, 64), 2)
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0, 0]))
    want = m.loopkv_read_tokens(kv, 0, 0, table, ints([64, 64]), ints([0, 0]), 64)
    err = ints([0])
    bad = table.clone()
    bad[0, 1] = kv.num_blocks
    got = m.loopkv_read_tokens(kv, 0, 0, bad, ints([64, 65]), ints([0, 0]), 64, err_flag=err)
    assert int(err) == m.LOOPKV_DEVERR_BLOCK_ID | m.LOOPKV_DEVERR_SEQ_LEN
    assert not got[0][1].any() and not got[1][1].any()
    assert not got[0][0, :32].any() and torch.equal(got[0][0, 32:], want[0][0, 32:])    # the keys' scales went with it
    assert torch.equal(got[1][0, :16], want[1][0, :16]) and not got[1][0, 16:32].any()


def attention_case(m, kind, d, heads, hkv, starts, lens, T, current, seed=0, scale=1.0, v_scale=1.0, sm_scale=1.0,
                   capacity=None, q_std=0.125):
    """Stores random tokens, attends a chunk and compares every row with the oracle."""
    B = len(starts)
    stored = [s + (0 if current else n) if s >= 0 else 0 for s, n in zip(starts, lens)]
    cap = capacity or max(1, max(stored))
    kv, table = cell_for(m, kind, B, hkv, d, cap, heads, seed=seed + 1)
    k, v = seeded_bf16((B, cap, hkv, d), seed + 2, scale), seeded_bf16((B, cap, hkv, d), seed + 3, v_scale)
    k[:, :, :, 3] *= 8
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0] * B), ints(stored))
    q = seeded_bf16((B, T, heads, d), seed + 4, q_std)
    cur = [seeded_bf16((B, T, hkv, d), seed + 5 + i, s) for i, s in enumerate((scale, v_scale))] if current else [None] * 2
    out = torch.full((B, T, heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    err = ints([0])
    m.loopkv_chunk_attention(kv, 0, 0, q, table, ints(starts), ints(lens), sm_scale, out, k_cur=cur[0], v_cur=cur[1],
                             err_flag=err)
    assert int(err) == 0
    g = heads // hkv
    for b in range(B):
        n = lens[b]
        assert (out[b, n:] == 7).all()
        if starts[b] < 0:
            assert not out[b, :n].any()
            continue
        for j in range(hkv):
            kh, vh = CO.stored_values(kind, host(k[b, :stored[b], j]), host(v[b, :stored[b], j]))
            if current:
                kh, vh = np.vstack([kh, host(cur[0][b, :n, j])]), np.vstack([vh, host(cur[1][b, :n, j])])
            for h in range(j * g, (j + 1) * g):
                want, slack = CO.chunk_attend(host(q[b, :n, h]), kh, vh, starts[b] + np.arange(n), sm_scale)
                off = np.abs(host(out[b, :n, h]) - want)
                assert np.all(off <= slack), (kind, b, h, float((off / np.maximum(slack, 1e-300)).max()))
    return kv, table, q, out


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("current", [False, True])
@pytest.mark.parametrize("heads,hkv", [(2, 2), (4, 2), (4, 1), (8, 1)])
def test_chunk_attention_short(m, kind, d, current, heads, hkv):
    attention_case(m, kind, d, heads, hkv, [0, 5, 31, 32, 95, -1, 64], [1, 3, 1, 2, 4, 4, 0], 4, current)


@pytest.mark.parametrize("kind", ["q4", "q2", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("current", [False, True])
def test_chunk_attention_long(m, kind, d, current):
    attention_case(m, kind, d, 4, 2, [0, 700, 129, 255], [300, 131, 128, 257], 300, current, seed=10)


@pytest.mark.parametrize("T,start", [(1, 0), (1, 1500), (16, 1000), (17, 1007), (33, 480), (64, 64), (65, 511), (127, 0),
                                     (128, 128), (129, 640), (256, 0), (257, 31), (513, 1)])
def test_chunk_attention_every_tile_edge(m, T, start):
    attention_case(m, "q4", 128, 2, 2, [start], [T], T, False, seed=T)
    attention_case(m, "q2", 64, 4, 1, [start], [T], T, True, seed=T + 1)


@pytest.mark.parametrize("kind", ["q4", "bf16"])
@pytest.mark.parametrize("scale,v_scale", [(1e-6, 1e-6), (1e-12, 1e12), (1.0, 1e5), (1e5, 1.0)])
def test_chunk_attention_scales(m, kind, scale, v_scale):
    """Keys and values far from one: the fp16 operands follow the data."""
    attention_case(m, kind, 128, 4, 2, [200, 0], [40, 33], 40, True, seed=3, scale=scale, v_scale=v_scale,
                   sm_scale=0.7 / scale)


def test_chunk_attention_peaked(m):
    """Logits of some hundred: a single key has all the weight."""
    attention_case(m, "q4", 128, 2, 2, [300], [70], 70, False, seed=8, q_std=8.0)
