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


# ---------------------------------------------------------------- together, and on the edges of what is allowed


def store(m, kind, B, hkv, d, capacity, heads, lens, seed=21):
    kv, table = cell_for(m, kind, B, hkv, d, capacity, heads, seed=seed)
    k, v = seeded_bf16((B, capacity, hkv, d), seed + 1), seeded_bf16((B, capacity, hkv, d), seed + 2)
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0] * B), ints(lens))
    return kv, table, k, v


def expect_rows(kind, k, v, stored, q, starts, lens, sm_scale, cur=None):
    """Oracle rows of every (sequence, head): [(b, h, rows, slack)]."""
    g = q.shape[2] // k.shape[2]
    found = []
    for b, (s, n) in enumerate(zip(starts, lens)):
        for j in range(k.shape[2]):
            kh, vh = CO.stored_values(kind, host(k[b, :stored[b], j]), host(v[b, :stored[b], j]))
            if cur is not None:
                kh, vh = np.vstack([kh, host(cur[0][b, :n, j])]), np.vstack([vh, host(cur[1][b, :n, j])])
            for h in range(j * g, (j + 1) * g):
                found.append((b, h, *CO.chunk_attend(host(q[b, :n, h]), kh, vh, s + np.arange(n), sm_scale)))
    return found


def check_rows(out, found):
    for b, h, want, slack in found:
        assert np.all(np.abs(host(out[b, :want.shape[0], h]) - want) <= slack), (b, h)


@pytest.mark.parametrize("hkv,heads", [(2, 2), (1, 4)])
def test_looped_chunk_step(m, hkv, heads):
    """Three ragged chunks through a plan of every kind: each cell's rows are the
    oracle's, from its own rotated and stored (or exact) keys."""
    L, N, B, d, cap = 2, 3, 3, 64, 260
    plan = ["q4", "reuse", "reuse", "q2", "bf16", "q4"]
    rng = np.random.default_rng(3)
    mb = -(-cap // 16)
    table = torch.from_numpy(rng.permutation(B * mb + 5)[: B * mb].reshape(B, mb).astype(np.int32)).cuda()
    kv = m.KVCells(plan, L, N, heads, d, B * mb + 5, B, mb, num_kv_heads=hkv)
    layers = [rotary_for(m, d, 64, False, True, seed=30 + 2 * j) for j in range(N)]
    start, err = ints([0, 0, 0]), ints([0])
    history = {c: [[], []] for c in range(6)}     # per cell: what the sequences' tokens are (k rotated, v)
    have = [0] * B
    T = 90
    for step, lens in enumerate([[90, 33, 1], [64, 90, 70], [1, 7, 90]]):
        rows = {c: fused_rows(B, T, heads, hkv, d, seed=1000 * step + c) for c in range(6)}
        q, k, v = ({c: rows[c][i] for c in range(6)} for i in range(3))
        out = {c: torch.zeros((B, T, heads, d), dtype=torch.bfloat16, device="cuda") for c in range(6)}
        chunk = m.LoopedChunkStep(kv, table, start, q, k, v, out, [x[0] for x in layers], 0.2, lens=ints(lens), err_flag=err)
        assert chunk.launches_per_step() == 12
        chunk.run()
        assert int(err) == 0
        turned = {}
        for c in range(6):
            _, qa, ka = layers[c % N]
            turned[c] = [[CO.norm_rope(host(x[c][b, :n]), have[b] + np.arange(n), **a) for b, n in enumerate(lens)]
                         for x, a in ((q, qa), (k, ka))]
        before = {c: [list(x) for x in history[c]] for c in range(6)}
        for c in range(6):
            history[c][0].append(turned[c][1])
            history[c][1].append([host(v[c][b, :n]) for b, n in enumerate(lens)])
        for c in range(6):
            src = c + 3 if plan[c] == "reuse" else c
            kept = before[src] if plan[c] == "reuse" else history[src]
            for b, n in enumerate(lens):
                kk, vv = (np.concatenate([x[b] for x in part] + [np.zeros((0, hkv, d), np.float32)]) for part in kept)
                for h in range(heads):
                    j = h * hkv // heads
                    kh, vh = CO.stored_values(plan[src], kk[:, j], vv[:, j])
                    if plan[c] == "reuse":
                        kh = np.vstack([kh, turned[c][1][b][:, j]])
                        vh = np.vstack([vh, host(v[c][b, :n, j])])
                    want, slack = CO.chunk_attend(turned[c][0][b][:, h], kh, vh, have[b] + np.arange(n), 0.2)
                    assert np.all(np.abs(host(out[c][b, :n, h]) - want) <= slack), (step, c, b, h)
        chunk.advance()
        have = [a + n for a, n in zip(have, lens)]
        assert start.tolist() == have


def test_chunk_then_decode_step(m):
    """The prompt side feeds the decode step: after a chunk, a decode step's
    stored cell attends over chunk and new token (checked against a chunk of one)."""
    B, H, d = 2, 4, 128
    kv, table, k, v = store(m, "q4", B, H, d, 100, H, [77, 64])
    q, kn, vn = (seeded_bf16((B, 1, H, d), 50 + i, 0.2) for i in range(3))
    start = ints([77, 64])
    m.loopkv_rope_append(kv, 0, 0, None, None, kn, vn, table, start)
    one = m.loopkv_chunk_attention(kv, 0, 0, q, table, start, sm_scale=0.5)
    dec = m.loopkv_decode_attention(kv, 0, 0, q[:, 0].contiguous(), table, start + 1, tau=0.0, sm_scale=0.5)
    full = [torch.cat([x, torch.zeros_like(x[:, :1])], 1) for x in (k, v)]
    for b, n in enumerate([77, 64]):
        full[0][b, n], full[1][b, n] = kn[b, 0], vn[b, 0]
    found = expect_rows("q4", *full, [78, 65], q, [77, 64], [1, 1], 0.5)
    check_rows(one, found)
    check_rows(dec[:, None], found)


@pytest.mark.parametrize("kind", ["q4", "bf16"])
@pytest.mark.parametrize("T", [3, 140])
def test_chunk_attention_device_faults(m, kind, T):
    """A bad block, a length beyond the bound and bad counts answer with zeros (or
    nothing) and a flag; the other sequences are as without them."""
    B, H, d, cap = 5, 2, 64, 400
    lens, starts = [T] * B, [200, 100, 250, 0, 31]
    kv, table, k, v = store(m, kind, B, H, d, cap, H, [s + T for s in starts])
    q = seeded_bf16((B, T, H, d), 9, 0.3)
    good = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints(starts), ints(lens))
    bad = table.clone()
    bad[1, 2], bad[4, 0] = kv.num_blocks, -1
    err = ints([0])
    out = torch.full_like(good, 7.0)
    m.loopkv_chunk_attention(kv, 0, 0, q, bad, ints(starts), ints([T, T, T, T + 1, T]), out=out, err_flag=err)
    assert int(err) == m.LOOPKV_DEVERR_BLOCK_ID | m.LOOPKV_DEVERR_SEQ_LEN
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    assert not out[1].any() and not out[4].any() and (out[3] == 7).all()
    err.zero_()
    # the bound also sizes the split of the context, so the same bits are those of the same bound
    ok = [s + T <= 249 for s in starts]
    good = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([s if f else -1 for s, f in zip(starts, ok)]), ints(lens),
                                    max_seq_len=249, err_flag=err)
    assert int(err) == 0 and not all(ok)
    out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints(starts), ints(lens), max_seq_len=249, err_flag=err)
    assert int(err) == m.LOOPKV_DEVERR_SEQ_LEN
    for b in range(B):
        assert torch.equal(out[b], good[b]) and bool(out[b].any()) == ok[b]


@pytest.mark.parametrize("kind,T", [("q4", 2), ("q2", 2), ("q4", 70)])
def test_chunk_attention_ignores_what_is_not_there(m, kind, T):
    """Stored bytes behind the last token, the open group's stale planes and the
    rows behind a chunk may hold anything, NaN included."""
    B, H, d, cap = 3, 2, 128, 160
    starts = [40, 64, 7]
    lens = [T, max(1, T - 1), 1]
    stored = [s + n for s, n in zip(starts, lens)]
    kv, table, k, v = store(m, kind, B, H, d, cap, H, stored)
    q = seeded_bf16((B, T, H, d), 9, 0.3)
    good = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints(starts), ints(lens))
    arena = kv.arena_view(0)
    before = arena.clone()
    ref, _, _, _ = store(m, kind, B, H, d, cap, H, stored)      # the bytes that are meant, over 0xFF elsewhere
    ref.arenas[0].fill_(0xFF)
    m.loopkv_rope_append(ref, 0, 0, None, None, k, v, table, ints([0] * B), ints(stored))
    arena.copy_(ref.arena_view(0))
    for b in range(B):
        kv.residuals[0][b, :, stored[b] % 32:] = float("nan")
        q[b, lens[b]:] = float("nan")
    assert not torch.equal(before, arena)
    again = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints(starts), ints(lens))
    assert torch.equal(again, good)
    got = m.loopkv_read_tokens(kv, 0, 0, table, ints(stored), ints([0] * B), cap)
    assert not torch.isnan(got[0]).any() and not torch.isnan(got[1]).any()


def test_shared_blocks_and_a_repeated_block(m):
    """Two sequences on the same blocks (a shared prefix), and one whose table
    names a block twice, are read as they are."""
    H, d = 2, 128
    kv, table, k, v = store(m, "q4", 2, H, d, 128, H, [128, 128])
    shared = table.clone()
    shared[1] = shared[0]
    q = seeded_bf16((2, 4, H, d), 3, 0.2)
    q[1] = q[0]
    out = m.loopkv_chunk_attention(kv, 0, 0, q, shared, ints([124, 124]))
    assert torch.equal(out[0], out[1])
    shared[1, 4:6] = shared[1, 0:2]          # keys 64 .. 95 are keys 0 .. 31 again
    out = m.loopkv_chunk_attention(kv, 0, 0, q, shared, ints([124, 124]))
    kk, vv = (torch.cat([x[0:1, :64], x[0:1, :32], x[0:1, 96:]], 1) for x in (k, v))
    check_rows(out[1:], expect_rows("q4", kk, vv, [128], q[1:], [124], [4], 1.0))


def test_calls_on_two_streams_at_once(m):
    """The same cell read by two streams while each has its own output, and two
    cells appended to at once."""
    B, H, d = 2, 4, 128
    kv, table, k, v = store(m, "q4", B, H, d, 600, H, [600, 555])
    other, _ = cell_for(m, "q4", B, H, d, 600, H)
    q = [seeded_bf16((B, T, H, d), T, 0.2) for T in (4, 200)]
    start = [ints([596, 551]), ints([400, 355])]
    want = [m.loopkv_chunk_attention(kv, 0, 0, x, table, s) for x, s in zip(q, start)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[torch.empty_like(w) for _ in range(10)] for w in want]
    for i in range(10):
        for j in range(2):
            m.loopkv_chunk_attention(kv, 0, 0, q[j], table, start[j], out=outs[j][i], stream=streams[j])
    m.loopkv_rope_append(other, 0, 0, None, None, k, v, table, ints([0, 0]), ints([600, 555]), stream=streams[2])
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, want[j]) for o in outs[j])
    same_cell(other, kv, [600, 555])


def test_captured_and_replayed_with_new_positions(m):
    """A captured pair of calls replays with the positions, lengths and rows that
    its buffers then hold."""
    B, H, d, T = 2, 2, 64, 5
    kv, table, k, v = store(m, "q4", B, H, d, 200, H, [0, 0])
    ref, _, _, _ = store(m, "q4", B, H, d, 200, H, [0, 0])
    r, _, _ = rotary_for(m, d, 64, True, True)
    q, kn, vn = (torch.zeros(B, T, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    start, lens, err = ints([-1, -1]), ints([T, T]), ints([0])
    qr, out = torch.zeros_like(q), torch.zeros_like(q)

    def both(cell, qr, out):
        m.loopkv_rope_append(cell, 0, 0, r, q, kn, vn, table, start, lens, qr, err_flag=err)
        m.loopkv_chunk_attention(cell, 0, 0, qr, table, start, lens, 0.3, out, err_flag=err)

    both(kv, qr, out)                        # skipped sequences: nothing is stored
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(kv, qr, out)
    have = [0, 0]
    for i in range(12):
        n = [1 + i % T, T - i % 3]
        for j, x in enumerate((q, kn, vn)):
            x.copy_(seeded_bf16((B, T, H, d), 100 * i + j))
        start.copy_(ints(have))
        lens.copy_(ints(n))
        graph.replay()
        qr2, out2 = torch.zeros_like(q), torch.zeros_like(q)
        both(ref, qr2, out2)
        for b in range(2):
            assert torch.equal(out[b, :n[b]], out2[b, :n[b]])
        have = [a + c for a, c in zip(have, n)]
        same_cell(kv, ref, have)
    assert int(err) == 0


def test_binding_refusals(m):
    kv, table, k, v = store(m, "q4", 2, 2, 64, 64, 2, [10, 10])
    q = seeded_bf16((2, 3, 2, 64), 1)
    s, r = ints([7, 7]), m.Rotary()
    ok = lambda **kw: m.loopkv_chunk_attention(kv, 0, 0, kw.pop("q", q), kw.pop("table", table), kw.pop("s", s), **kw)  # noqa: E731
    ok()
    for kw, text in ((dict(q=q.float()), "bfloat16"), (dict(q=q[:, :, :1]), "shape"), (dict(q=q.transpose(2, 3)), "shape"),
                     (dict(s=s.long()), "int32"), (dict(s=s[:1]), "shape"), (dict(table=table[:, :2]), "shape"),
                     (dict(out=q), "overlaps q"), (dict(k_cur=q), "together"), (dict(out=torch.empty_like(q).transpose(1, 2)), "out"),
                     (dict(q=seeded_bf16((2, 3, 2, 65), 1)[..., 1:]), "multiples of 8"), (dict(new_lens=s.cpu()), "CUDA")):
        with pytest.raises(ValueError, match=text):
            ok(**kw)
    with pytest.raises(m.LoopKVError):
        ok(max_seq_len=65)
    with pytest.raises(ValueError, match="overlaps k_new"):
        m.loopkv_rope_append(kv, 0, 0, r, q, q, v[:, :3], table, s, q_out=q)
    with pytest.raises(ValueError, match="rotary"):
        m.loopkv_rope_append(kv, 0, 0, None, q, k[:, :3], v[:, :3], table, s)
    with pytest.raises(ValueError, match="entries"):
        m.loopkv_norm_rope(m.Rotary(q_weight=seeded_bf16((128,), 1)), q, None, s)
    with pytest.raises(ValueError, match="overlaps"):
        m.loopkv_read_tokens(kv, 0, 0, table, s, s, 3, k_out=q, v_out=q)
    with pytest.raises(ValueError, match="no cell"):
        m.loopkv_read_tokens(kv, 1, 0, table, s, s, 3)
    with pytest.raises(ValueError, match="no storage"):
        m.loopkv_read_tokens(m.KVCells(["q4", "q4"], 1, 2, 2, 64, 8, 2, 4, allocate={0}), 0, 1, table, s, s, 3)


def test_empty_chunks(m):
    kv, table, k, v = store(m, "q4", 2, 2, 64, 64, 2, [10, 10])
    q, s = seeded_bf16((2, 0, 2, 64), 1), ints([10, 10])
    assert m.loopkv_chunk_attention(kv, 0, 0, q, table, s).shape == q.shape
    m.loopkv_rope_append(kv, 0, 0, m.Rotary(), q, q, q, table, s)
    assert m.loopkv_norm_rope(m.Rotary(), q, q, s)[1].shape == q.shape
    assert m.loopkv_read_tokens(kv, 0, 0, table, s, s, 0)[0].shape == q.shape
    none = ints([])
    x = seeded_bf16((0, 4, 2, 64), 1)
    assert m.loopkv_chunk_attention(kv, 0, 0, x, table[:0], none).shape == x.shape


@pytest.mark.parametrize("kind", ["q4", "q2"])
def test_long_context(m, kind):
    """Context longer than the decode kernel's limit, and offsets into an arena
    of more than 2^31 bytes."""
    d, n, T = 128, 70_000, 3
    rec = m.loopkv_record_bytes(d, kind)
    pool = 2**31 // rec + 6000
    mb = -(-n // 16)
    kv = m.KVCells([kind], 1, 1, 1, d, pool, 1, mb)
    table = torch.arange(pool - 1, pool - 1 - mb, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    k, v = seeded_bf16((1, n, 1, d), 1), seeded_bf16((1, n, 1, d), 2)
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0]))
    q = seeded_bf16((1, T, 1, d), 3, 0.4)
    out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([n - T]))
    check_rows(out, expect_rows(kind, k, v, [n], q, [n - T], [T], 1.0))
    wide = seeded_bf16((1, 150, 1, d), 4, 0.4)
    out = m.loopkv_chunk_attention(kv, 0, 0, wide, table, ints([n - 150]))
    check_rows(out[:, ::37], [(b, h, w[::37], e[::37]) for b, h, w, e in
                              expect_rows(kind, k, v, [n], wide, [n - 150], [150], 1.0)])


def test_zero_and_negative_scales(m):
    """sm_scale 0 weighs all visible keys alike; a negative one turns the order."""
    B, H, d = 1, 2, 64
    kv, table, k, v = store(m, "q4", B, H, d, 100, H, [100])
    for T in (2, 40):
        q = seeded_bf16((B, T, H, d), 5)
        for sm in (0.0, -0.4):
            out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([100 - T]), sm_scale=sm)
            check_rows(out, expect_rows("q4", k, v, [100], q, [100 - T], [T], sm))


@pytest.mark.parametrize("kind", ["q4", "bf16"])
@pytest.mark.parametrize("T", [3, 150])
def test_rows_behind_a_current_chunk_are_not_read(m, kind, T):
    B, H, d = 2, 2, 128
    kv, table, k, v = store(m, kind, B, H, d, 64, H, [50, 0])
    q, kc, vc = (seeded_bf16((B, T, H, d), 60 + i, 0.4) for i in range(3))
    start, lens = ints([50, 0]), ints([T - 1, 2])
    good = m.loopkv_chunk_attention(kv, 0, 0, q, table, start, lens, k_cur=kc, v_cur=vc)
    for x in (q, kc, vc):
        for b, n in enumerate([T - 1, 2]):
            x[b, n:] = float("nan")
    again = m.loopkv_chunk_attention(kv, 0, 0, q, table, start, lens, k_cur=kc, v_cur=vc)
    assert torch.equal(good, again) and not torch.isnan(again).any()


@pytest.mark.parametrize("T", [5, 140])
def test_outlier_channels_of_exact_keys(m, T):
    """Keys with a channel 2^12 times the others, as open groups, bf16 cells and
    current rows hold them exactly: the logits keep the small channels whole."""
    B, H, d, n = 1, 2, 64, 100
    kv, table = cell_for(m, "bf16", B, H, d, n)
    k, v = seeded_bf16((B, n, H, d), 1), seeded_bf16((B, n, H, d), 2)
    kc, vc = seeded_bf16((B, T, H, d), 3), seeded_bf16((B, T, H, d), 4)
    q = seeded_bf16((B, T, H, d), 5, 0.3)
    k[..., 7] *= 4096
    kc[..., 7] *= 4096
    q[..., 7] *= 2.0**-12
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0]))
    out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([n]), k_cur=kc, v_cur=vc)
    check_rows(out, expect_rows("bf16", k, v, [n], q, [n], [T], 1.0, cur=(kc, vc)))


@pytest.mark.parametrize("kind", ["q4", "q2"])
@pytest.mark.parametrize("B,H,d,n", [(1, 4, 128, 3000), (1, 16, 128, 2500), (10, 16, 64, 1200), (40, 16, 128, 300),
                                     (13, 16, 128, 500), (64, 4, 64, 1500)])
def test_few_rows_at_every_cta_size(m, kind, B, H, d, n):
    """Grids from four pairs of sequence and head to some hundred: other CTA
    sizes and splits of the context for each."""
    lens = [n - 7 * (b % 5) for b in range(B)]
    T = 3
    kv, table, k, v = store(m, kind, B, H, d, n, H, lens)
    q = seeded_bf16((B, T, H, d), 3, 0.3)
    err = ints([0])
    out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([x - T for x in lens]), err_flag=err)
    assert int(err) == 0
    some = sorted({0, B // 2, B - 1})
    check_rows(out[some], expect_rows(kind, k[some], v[some], [lens[b] for b in some], q[some],
                                      [lens[b] - T for b in some], [T] * len(some), 1.0))


def test_new_outputs_belong_to_the_stream_of_the_call(m):
    """A new output is filled on the stream that the call goes to: work that the
    current stream still has before it does not come after the result."""
    B, H, d = 2, 2, 64
    kv, table, k, v = store(m, "q4", B, H, d, 64, H, [40, 33])
    q, s, lens, r = seeded_bf16((B, 4, H, d), 3), ints([36, 29]), ints([4, 3]), m.Rotary()
    stored, skip = ints([40, 33]), ints([-1, -1])
    calls = [lambda **kw: m.loopkv_chunk_attention(kv, 0, 0, q, table, s, lens, **kw),
             lambda **kw: m.loopkv_norm_rope(r, q, None, s, lens, **kw)[0],
             lambda **kw: m.loopkv_read_tokens(kv, 0, 0, table, stored, s, 4, **kw)[1],
             lambda **kw: m.loopkv_rope_append(kv, 0, 0, r, q, k[:, :4], v[:, :4], table, skip, **kw)]
    want = [c() for c in calls]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        torch.cuda._sleep(20_000_000)
        got = c(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, w)


@pytest.mark.parametrize("kind", ["q4", "bf16"])
@pytest.mark.parametrize("T", [4, 130])
def test_zero_values_and_values_of_far_apart_sizes(m, kind, T):
    """Most blocks' values are exactly zero, or 2^-40 of the others: they still
    take their weights out of the rest."""
    B, H, d, n = 1, 2, 128, 1600
    kv, table = cell_for(m, kind, B, H, d, n)
    k, v = seeded_bf16((B, n, H, d), 1), seeded_bf16((B, n, H, d), 2)
    v[:, 64:1200] = 0
    v[:, 1200:1500] *= 2.0**-40
    m.loopkv_rope_append(kv, 0, 0, None, None, k, v, table, ints([0]))
    q = seeded_bf16((B, T, H, d), 3, 1.0)
    out = m.loopkv_chunk_attention(kv, 0, 0, q, table, ints([n - T]))
    step = max(1, T // 5)
    check_rows(out[:, ::step], [(b, h, w[::step], e[::step]) for b, h, w, e in
                                expect_rows(kind, k, v, [n], q, [n - T], [T], 1.0)])


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("d,interleaved", [(64, False), (128, True)])
def test_norm_of_one_side_only(m, which, d, interleaved):
    """A weight for queries or for keys alone, heads of both in one thread's item."""
    table = CO.rope_angles(40, d)
    w = seeded_bf16((d,), 7, 0.2) + 1
    r = m.Rotary(torch.from_numpy(table).cuda(), interleaved=interleaved, eps=1e-5, **{which + "_weight": w})
    q, k, v = fused_rows(2, 9, 3, 3, d, seed=5)
    start = ints([0, 20])
    q_out, k_out = m.loopkv_norm_rope(r, q, k, start)
    for x, o, name in ((q, q_out, "q"), (k, k_out, "k")):
        for b, s in enumerate([0, 20]):
            want = CO.norm_rope(host(x[b]), s + np.arange(9), table, interleaved, host(w) if name == which else None, 1e-5)
            assert np.array_equal(host(o[b]), want)
    kv, bt = cell_for(m, "bf16", 2, 3, d, 40)
    got = m.loopkv_rope_append(kv, 0, 0, r, q, k, v, bt, start)
    assert torch.equal(got, q_out)
    kk, vv = m.loopkv_read_tokens(kv, 0, 0, bt, ints([9, 29]), start, 9)
    assert torch.equal(kk, k_out) and torch.equal(vv, v.contiguous())
