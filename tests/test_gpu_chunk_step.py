"""LoopedChunkStep on the edges of what it is given: sequences that do not fit,
streams, and drafted tokens that are rejected."""

import pytest
import torch

from loopkv_testlib import seeded_bf16
from oracle import chunk_oracle as CO
from test_gpu_chunk import fused_rows, host, ints

pytestmark = pytest.mark.gpu

PLAN, L, N = ["q4", "reuse", "bf16", "q2", "q4", "bf16"], 2, 3


@pytest.fixture(scope="module")
def m():
    import mixed_precision_kv_loopkv_b200 as pkg
    return pkg


def make(m, B, T, capacity, positions, heads=4, hkv=2, d=64, seed=0, plan=PLAN, **kw):
    """Cells, start, outputs (filled with 7) and a step over seeded rows."""
    mb = capacity // 16
    kv = m.KVCells(plan, L, N, heads, d, B * mb, B, mb, num_kv_heads=hkv)
    table = torch.arange(B * mb, dtype=torch.int32, device="cuda").view(B, mb)
    rotary = m.Rotary(m.rope_table(positions, d), k_weight=seeded_bf16((d,), 5, 0.2) + 1)
    start = ints([0] * B)
    return kv, start, step_over(m, kv, table, start, T, rotary, seed, **kw)


def step_over(m, kv, table, start, T, rotary, seed, **kw):
    B = start.shape[0]
    rows = {c: fused_rows(B, T, kv.num_heads, kv.num_kv_heads, kv.head_dim, seed + c) for c in range(6)}
    q, k, v = ({c: rows[c][i] for c in range(6)} for i in range(3))
    out = {c: torch.full((B, T, kv.num_heads, kv.head_dim), 7.0, dtype=torch.bfloat16, device="cuda") for c in range(6)}
    return m.LoopedChunkStep(kv, table, start, q, k, v, out, rotary, 0.3, **kw)


@pytest.mark.parametrize("reuse", [True, False])
@pytest.mark.parametrize("positions", [100, 160, 165])
def test_a_sequence_past_its_rotation_table(m, positions, reuse):
    """Where the table (or the cell) ends before the chunk does, no cell answers for
    the sequence or stores of it, and it is not moved on; the others are as ever."""
    B, T, cap = 4, 10, 160
    plan = PLAN if reuse else ["q4", "q2", "bf16", "q2", "q4", "bf16"]
    limit = min(positions, cap)
    have = [0, limit - 20, limit - 5, limit - 9]
    lens = [10, 10, 10, 9]
    err = ints([0])
    kv, start, step = make(m, B, T, cap, positions, plan=plan, lens=ints(lens), err_flag=err)
    ref_kv, ref_start, ref = make(m, B, T, cap, 400, plan=plan, lens=ints(lens))
    for s, seed in ((step, 50), (ref, 50)):     # something is stored before
        fill = step_over(m, s.kv, s.block_table, ints([0] * B), 155, m.Rotary(), seed, lens=ints(have))
        fill.run()
    start.copy_(ints(have))
    ref_start.copy_(ints([have[0], have[1], -1, have[3]]))
    for name in step._rows:
        step._rows[name].fill_(float("nan"))
    before = [None if a is None else a.clone() for a in kv.arenas]
    step.run()
    ref.run()
    assert int(err) == m.LOOPKV_DEVERR_SEQ_LEN
    for c in range(6):
        assert torch.equal(step.out[c], ref.out[c]) and not step.out[c][2].any()
        if kv.arenas[c] is not None:
            a, b = kv.arena_view(c), before[c].view_as(kv.arena_view(c))
            assert torch.equal(a[step.block_table[2].long()], b[step.block_table[2].long()])
    step.advance()
    assert start.tolist() == [10, limit - 10, limit - 5, limit]


def test_lengths_that_are_none_do_not_move_a_sequence(m):
    lens, err = ints([11, -3, 0, 10]), ints([0])
    kv, start, step = make(m, 4, 10, 160, 200, lens=lens, err_flag=err)
    start.copy_(ints([5, 5, 500, -1]))
    step.run()
    step.advance()
    assert start.tolist() == [5, 5, 500, -1] and int(err) == m.LOOPKV_DEVERR_SEQ_LEN
    assert all((o[:3] == 7).all() and not o[3].any() for o in step.out.values())


def test_all_tokens_without_lengths(m):
    err = ints([0])
    kv, start, step = make(m, 3, 10, 64, 40, err_flag=err)
    start.copy_(ints([30, 31, -1]))
    step.run()
    assert int(err) == m.LOOPKV_DEVERR_SEQ_LEN
    step.advance()
    assert start.tolist() == [40, 31, -1]
    assert all(o[0].any() and not o[1:].any() for o in step.out.values())


def test_run_and_advance_on_another_stream(m):
    """Steps on a stream that has work before them: positions move when the calls
    before have read them."""
    B, T = 3, 10
    want_kv, want_start, want = make(m, B, T, 160, 400)
    kv, start, step = make(m, B, T, 160, 400)
    outs = []
    for _ in range(4):
        want.run()
        outs.append({c: o.clone() for c, o in want.out.items()})
        want.advance()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    for i in range(4):
        step.run(stream=side)
        if i < 3:
            step.advance()
    side.synchronize()
    assert start.tolist() == [30] * B and want_start.tolist() == [40] * B
    for c in range(6):
        assert torch.equal(step.out[c], outs[3][c])
        if kv.arenas[c] is not None:
            assert torch.equal(kv.arenas[c], want_kv.arenas[c])


@pytest.mark.parametrize("d,hkv", [(64, 2), (128, 4)])
def test_drafted_tokens_are_checked_then_stored(m, d, hkv):
    """Rounds of drafted tokens over key group borders: every row is the oracle's
    over what was accepted before and its own draft, and the cells hold what they
    would hold if no other token had ever been seen."""
    B, T, H = 3, 20, 4
    lens, err = ints([T] * B), ints([0])
    kv, start, step = make(m, B, T, 160, 400, d=d, hkv=hkv, lens=lens, err_flag=err)
    ref_kv, ref_start, ref = make(m, B, T, 160, 400, d=d, hkv=hkv, lens=ints([0] * B))
    rotary, have = step.rotary[0], [0] * B
    kept = {c: [[[], []] for _ in range(B)] for c in range(6)}     # rotated keys and values of the accepted
    weight = host(rotary.k_weight)
    table = host(rotary.table)
    for turn, (drafted, accepted) in enumerate([([20, 17, 20], [20, 17, 3]), ([20, 20, 5], [13, 1, 5]), ([9, 20, 20], [0, 15, 20]),
                                                ([20, 20, 20], [1, 14, 7]), ([20, 1, 20], [11, 1, 19])]):
        for c in range(6):
            x = fused_rows(B, T, H, hkv, d, 1000 * turn + c)
            for s in (step, ref):
                s.q[c], s.k[c], s.v[c] = x
        lens.copy_(ints(drafted))
        before = [None if a is None else a.clone() for a in kv.arenas]
        step.run(store=False)
        assert all(a is None or torch.equal(a, b) for a, b in zip(kv.arenas, before))
        for c in range(6):
            src = c + N if PLAN[c] == "reuse" else c
            for b, n in enumerate(drafted):
                pos = have[b] + torch.arange(n).numpy()
                qr = CO.norm_rope(host(step.q[c][b, :n]), pos, table)
                kr = CO.norm_rope(host(step.k[c][b, :n]), pos, table, weight=weight)
                for h in range(H):
                    j = h * hkv // H
                    old = [torch.cat([torch.zeros(0, hkv, d)] + x).numpy()[:, j] for x in kept[src][b]]
                    kh, vh = CO.stored_values(PLAN[src], *old)
                    kh = torch.cat([torch.from_numpy(kh), torch.from_numpy(kr[:, j]).double()]).numpy()
                    vh = torch.cat([torch.from_numpy(vh), step.v[c][b, :n, j].cpu().double()]).numpy()
                    want, slack = CO.chunk_attend(qr[:, h], kh, vh, pos, 0.3)
                    assert (abs(host(step.out[c][b, :n, h]) - want) <= slack).all(), (turn, c, b, h)
        for c in range(6):
            for b, n in enumerate(accepted):
                pos = have[b] + torch.arange(n).numpy()
                kept[c][b][0].append(torch.from_numpy(CO.norm_rope(host(step.k[c][b, :n]), pos, table, weight=weight)))
                kept[c][b][1].append(step.v[c][b, :n].float().cpu())
        for x in (lens, ref.lens):
            x.copy_(ints(accepted))
        step.store()
        step.advance()
        ref.run()
        ref.advance()
        have = [a + n for a, n in zip(have, accepted)]
        assert start.tolist() == have == ref_start.tolist()
        for c in range(6):
            if kv.arenas[c] is not None:
                assert torch.equal(kv.arenas[c], ref_kv.arenas[c])
                if kv.residuals[c] is not None:
                    for b, n in enumerate(have):
                        assert torch.equal(kv.residuals[c][b, :, : n % 32], ref_kv.residuals[c][b, :, : n % 32])
    assert int(err) == 0


def test_how_far_a_cell_can_go_back(m):
    """A quantised cell appended to again from the last multiple of 32 tokens on,
    a bf16 cell from anywhere, holds what it would hold without the rejected tokens."""
    rows = [fused_rows(1, 100, 4, 2, 64, seed) for seed in (1, 2)]
    for kind, back in (("q4", 64), ("q4", 70), ("q2", 64), ("bf16", 3), ("bf16", 50)):
        got, want = (m.KVCells([kind], 1, 1, 4, 64, 8, 1, 8, num_kv_heads=2) for _ in range(2))
        table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
        (_, k1, v1), (_, k2, v2) = rows

        def append(kv, k, v, at, lo, hi):
            m.loopkv_rope_append(kv, 0, 0, None, None, k[:, lo:hi], v[:, lo:hi], table, ints([at]))

        append(got, k1, v1, 0, 0, 75)
        append(got, k2, v2, back, 0, 40)
        append(want, k1, v1, 0, 0, back)
        append(want, k2, v2, back, 0, 40)
        n = back + 40
        for a, b in zip(*(m.loopkv_read_tokens(kv, 0, 0, table, ints([n]), ints([0]), n) for kv in (got, want))):
            assert torch.equal(a, b), (kind, back)


def test_prefill_on_another_stream(m):
    """The rows that prefill copies and the positions that it makes are read when
    they are there, on a stream that is behind and beside one that is busy."""
    k, v = seeded_bf16((3, 90, 2, 64), 1), seeded_bf16((3, 90, 2, 64), 2)
    kvs = [m.KVCells(["q4"], 1, 1, 2, 64, 24, 3, 8) for _ in range(2)]
    table = torch.arange(24, dtype=torch.int32, device="cuda").view(3, 8)
    lens = [90, 33, 70]
    m.prefill(kvs[0], 0, 0, k, v, table, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)          # the current stream's own work
    m.prefill(kvs[1], 0, 0, k, v, table, lens, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kvs[0].arenas[0], kvs[1].arenas[0])


def test_a_captured_step_replays_chunk_after_chunk(m):
    """run and advance in one graph: each replay is the next chunk of what its
    buffers then hold."""
    B, T = 3, 12
    lens, err = ints([T] * B), ints([0])
    kv, start, step = make(m, B, T, 160, 160, lens=lens, err_flag=err)
    ref_kv, ref_start, ref = make(m, B, T, 160, 160, lens=ints([T] * B))
    start.fill_(-1)
    step.run()                               # warm-up: every sequence is skipped
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
        step.advance()
    start.fill_(0)
    for turn, n in enumerate([[12, 1, 7], [12, 12, 0], [5, 12, 12], [12, 12, 12], [1, 2, 12]]):
        for x in (lens, ref.lens):
            x.copy_(ints(n))
        for c in range(6):
            x = fused_rows(B, T, 4, 2, 64, 100 * turn + c)
            for held, new in zip((step.q[c], step.k[c], step.v[c]), x):
                held.copy_(new)
            ref.q[c], ref.k[c], ref.v[c] = x
        graph.replay()
        ref.run()
        ref.advance()
        assert start.tolist() == ref_start.tolist()
        for c in range(6):
            for b in range(B):
                assert torch.equal(step.out[c][b, : n[b]], ref.out[c][b, : n[b]])
            assert kv.arenas[c] is None or torch.equal(kv.arenas[c], ref_kv.arenas[c])
    assert int(err) == 0
