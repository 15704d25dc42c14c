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
