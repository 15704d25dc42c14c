"""Which stream the steps' own operations go to (no kernel is launched)."""

import contextlib

import pytest
import torch


@pytest.fixture()
def step_module(monkeypatch):
    """The step module with its calls recorded, and the stream of each torch operation on the positions."""
    from mixed_precision_kv_loopkv_b200 import step
    for name in ("loopkv_norm_rope", "loopkv_rope_append", "loopkv_chunk_attention", "loopkv_quantize_append",
                 "loopkv_decode_attention", "loopkv_append_decode_attention"):
        monkeypatch.setattr(step, name, lambda *a, **kw: None)
    used = []

    @contextlib.contextmanager
    def on(stream):
        used.append(stream)
        yield

    monkeypatch.setattr(step, "_on", on)
    return step, used


class Cells:
    num_layers, plan_codes, max_blocks_per_seq, block_size, num_heads, num_kv_heads = 1, [0], 4, 16, 1, 1


def steps(step):
    x = {0: torch.zeros(2, 3, 1, 64, dtype=torch.bfloat16)}
    rotary = step.Rotary()
    start = torch.tensor([0, -1], dtype=torch.int32)
    pos = torch.tensor([5, 6], dtype=torch.int32)
    chunk = step.LoopedChunkStep(Cells(), None, start, x, x, x, x, rotary, 1.0)
    decode = step.LoopedDecodeStep(Cells(), None, pos, x, x, x, x, 0.0, 1.0, 64)
    return (chunk, start, [3, -1]), (decode, pos, [6, 7])


@pytest.mark.parametrize("which", [0, 1])
def test_advance_follows_the_stream_of_the_run(step_module, which):
    step, used = step_module
    x, positions, moved = steps(step)[which]
    x.run(stream="side")
    x.advance()
    assert used == ["side"] and positions.tolist() == moved
    x.advance(stream="other")
    x.run()
    x.advance()
    assert used == ["side", "other", None]


def test_prefill_copies_on_the_stream_of_its_appends(step_module):
    step, used = step_module
    k = torch.zeros(2, 9, 1, 64, dtype=torch.bfloat16)
    step.prefill(Cells(), 0, 0, k, k, None, [9, 4], stream="side")
    assert used == ["side", "side"]
