"""The prompt-side operators of a LoopKV cell, case by case: what is measured, and their plain forms.

Four operators of one path, a chunk of new tokens through a (loop, layer) cell:
  norm_rope   norms of queries and keys for each head, with the position rotation in the same pass;
  append      keys (normed, rotated) and values appended to a paged 4-bit, 2-bit or bf16 cell, queries
              rotated on the way, and the cell's tokens read back as the values that they stand for;
  read        a range of a cell's tokens read back;
  chunk       attention of a chunk of new tokens over a paged cell, the chunk's own tokens stored in it
              ("stored") or given as exact rows beside it ("current", a reuse cell's form).

Definitions that both sides keep to.  Rotation and norm: with r = fp32(1 / sqrt(mean(x^2) + eps)) from a
64-bit mean, a = (x r) w and y1 = a1 cos - a2 sin, y2 = a2 cos + a1 sin, every product and sum one rounded
fp32 operation, then one rounding to bf16.  Quantiser: s = bf16((max - min) / (2^b - 1)),
code = rint((x - min) / s); keys per channel over 32 tokens, values per token over 32 channels; keys of an
unfinished group of 32 stay exact.  Codes are decided by a border, so the steps are part of the definition.
"""

import math

import torch

own = False

GROUP, BLOCK, EPS = 32, 16, 1e-6
BITS = {"q4": 4, "q2": 2}


def listed():
    return [
        # every token of a decode batch, all heads of one layer: a few microseconds, launch latency counts
        dict(name="norm_rope decode batch", op="norm_rope", batch=64, tokens=1, heads=16, kv_heads=16, dim=128, rot=128,
             pairs="halves", norm=True, context=8192, ragged=False),
        # the reuse cells of a prompt chunk: queries and keys of some thousand tokens, grouped heads, partial rotation
        dict(name="norm_rope prompt", op="norm_rope", batch=3, tokens=2731, heads=32, kv_heads=8, dim=64, rot=32,
             pairs="neighbours", norm=True, context=8192, ragged=True),
        # a decode step's store: one token for each sequence, at any place of its open group
        dict(name="append one token", op="append", kind="q4", batch=64, tokens=1, heads=16, kv_heads=16, dim=128, rot=128,
             pairs="halves", norm=True, context=2048, ragged=False),
        # a whole prompt into an empty 4-bit cell
        dict(name="append prompt", op="append", kind="q4", batch=1, tokens=8191, heads=16, kv_heads=16, dim=128, rot=128,
             pairs="halves", norm=False, context=0, ragged=False),
        # a ragged batch of prompt chunks into a 2-bit cell with grouped heads
        dict(name="append ragged chunks", op="append", kind="q2", batch=8, tokens=517, heads=16, kv_heads=4, dim=64, rot=64,
             pairs="neighbours", norm=True, context=2048, ragged=True),
        # one sequence's last open groups, as a scheduler moves them
        dict(name="read tail", op="read", kind="q2", batch=4, tokens=77, heads=4, kv_heads=4, dim=64, context=1000, ragged=True),
        # a long prefix taken out of a 4-bit cell
        dict(name="read prefix", op="read", kind="q4", batch=4, tokens=8192, heads=16, kv_heads=16, dim=128, context=8192, ragged=True),
        # the check of a few drafted tokens for every sequence of a batch
        dict(name="chunk of 4, batch 32", op="chunk", mode="stored", kind="q4", batch=32, tokens=4, heads=16, kv_heads=16, dim=128,
             context=4096, ragged=False),
        # two short sequences: launch latency and the walk over the context
        dict(name="chunk of 7, short", op="chunk", mode="stored", kind="q2", batch=2, tokens=7, heads=8, kv_heads=2, dim=64,
             context=333, ragged=True),
        # a prompt's last chunk over all that is stored before it
        dict(name="chunk of 2048 at 16K", op="chunk", mode="stored", kind="q4", batch=1, tokens=2048, heads=16, kv_heads=16, dim=128,
             context=14336, ragged=False),
        # a reuse cell in a prompt: the final loop's cell and the chunk's own exact rows
        dict(name="chunk of 512, reuse cell", op="chunk", mode="current", kind="q4", batch=4, tokens=512, heads=16, kv_heads=16,
             dim=128, context=2048, ragged=True),
        # a ragged batch with grouped heads over an unquantised cell
        dict(name="chunk of 301, grouped, bf16", op="chunk", mode="stored", kind="bf16", batch=6, tokens=301, heads=16, kv_heads=4,
             dim=128, context=1500, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "read", "chunk", "chunk"))
    dim = rng.choice((64, 128))
    kv_heads = rng.choice((2, 4, 5, 8, 16))
    heads = kv_heads * rng.choice((1, 2, 4) if kv_heads <= 8 else (1,))
    kind = rng.choice(("q4", "q2", "bf16"))
    c = dict(op=op, batch=1, tokens=1, heads=heads, kv_heads=kv_heads, dim=dim, ragged=rng.random() < 0.6)
    if op in ("norm_rope", "append"):
        c.update(rot=rng.choice((dim, dim // 2)), pairs=rng.choice(("halves", "neighbours")), norm=rng.random() < 0.6)
    if op == "norm_rope":
        c.update(tokens=_log(rng, 1, 4000), context=_log(rng, 1, 16000))
        c["batch"] = _log(rng, 1, max(1, min(64, 8000 // c["tokens"])))
    elif op == "append":
        c.update(kind=kind, tokens=1 if rng.random() < 0.3 else _log(rng, 2, 4000), context=_log(rng, 32, 4000))
        c["batch"] = _log(rng, 1, max(1, min(64, 6000 // c["tokens"])))
    elif op == "read":
        c.update(kind=kind, tokens=_log(rng, 1, 8000))
        c["context"] = c["tokens"] + rng.randint(0, 3000)
        c["batch"] = _log(rng, 1, max(1, min(16, 24000 // c["context"])))
    else:
        c.update(kind=kind, mode=rng.choice(("stored", "current")), tokens=_log(rng, 1, 1500), context=_log(rng, 1, 8000))
        span = c["context"] + c["tokens"]
        c["batch"] = _log(rng, 1, max(1, min(32, 40000 // span, 2048 * 15360 * 16 // (c["tokens"] * span * heads))))
    return c


# ----------------------------------------------------------------- inputs


def _lengths(case, seed):
    """Stored tokens before the chunk, and new tokens, of every sequence."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    b, t, n = case["batch"], case["tokens"], case["context"]
    pick = lambda lo, hi: torch.randint(lo, hi + 1, (b,), generator=g)  # noqa: E731
    new = torch.full((b,), t)
    if case["ragged"]:
        new = pick(max(1, t // 3), t)
        new[0] = t
    before = pick(n // 2, n) if case["ragged"] else torch.full((b,), n)
    if case["op"] == "append":
        # The appended place is written again by the next pass over the same state, so the exact keys of
        # the open group that a pass starts from must outlive it: one token anywhere, chunks from a group's start.
        before = pick(n // 2, n) if t == 1 else before // GROUP * GROUP
    return before, new


def _random(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def _kv(case, tokens, seed):
    """bf16 keys (four channels of each head ten times as large) and values [B, tokens, Hkv, D]."""
    shape = (case["batch"], tokens, case["kv_heads"], case["dim"])
    k, v = _random(shape, seed), _random(shape, seed + 1)
    far = torch.argsort(_random(shape[2:], seed + 2), dim=-1)[:, :4]
    k *= torch.ones(shape[2:], device="cuda").scatter_(1, far, 10.0)
    return k.bfloat16(), v.bfloat16()


def _quantise(x, bits, dim):
    """Codes, scale and minimum of the groups along `dim`, fp32."""
    low, high = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    scale = ((high - low) / (2**bits - 1)).bfloat16().float()
    code = torch.where(scale > 0, torch.round((x - low) / scale), torch.zeros_like(x)).clamp_(0, 2**bits - 1)
    return code, scale, low


def _plane(code2):
    """2-bit codes [..., D] -> bytes [..., D / 4], the first of four channels in the lowest bits."""
    c = code2.unflatten(-1, (-1, 4))
    return c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6)


def _paged(x):
    """[B, S, H, n] -> [B, S / 16, H, 16, n]."""
    return x.unflatten(1, (-1, BLOCK)).transpose(2, 3)


def _bytes(x):
    return x.contiguous().view(torch.uint8).flatten(3)


def _records(kind, k, v):
    """Records uint8 [B, S / 16, Hkv, record] of S tokens (a multiple of 32), laid out as the cells store them."""
    if kind == "bf16":
        return torch.cat([_bytes(_paged(k)), _bytes(_paged(v))], dim=-1)
    bits, d = BITS[kind], k.shape[-1]
    kc, ks, km = _quantise(k.float().unflatten(1, (-1, GROUP)), bits, 2)
    kc = kc.flatten(1, 2).to(torch.uint8)
    meta = torch.stack([ks[:, :, 0], km[:, :, 0]], -1).bfloat16()                  # [B, S / 32, H, D, 2]
    meta = meta.unflatten(3, (2, d // 2)).movedim(3, 2).flatten(1, 2)              # [B, S / 16, H, D / 2, 2]
    del ks, km
    vc, vs, vm = _quantise(v.float().unflatten(3, (-1, GROUP)), bits, 4)
    vc = vc.flatten(3, 4).to(torch.uint8)
    vmeta = _paged(torch.stack([vs[..., 0], vm[..., 0]], -1).bfloat16().flatten(3, 4))
    if kind == "q4":
        parts = [_paged(_plane(kc >> 2)), _paged(_plane(kc & 3)), meta, _paged(_plane(vc >> 2)).transpose(3, 4), vmeta,
                 _paged(_plane(vc & 3))]
    else:
        parts = [_paged(_plane(kc)), meta, _paged(_plane(vc)).transpose(3, 4), vmeta]
    return torch.cat([_bytes(p) for p in parts], dim=-1)


def _cell(case, stored, capacity, seed):
    """A cell that holds stored[b] tokens and has room for `capacity`: arena, table, open keys."""
    b, h, d, kind = case["batch"], case["kv_heads"], case["dim"], case["kind"]
    blocks = -(-capacity // GROUP) * 2
    g = torch.Generator().manual_seed(seed * 7 + 2)
    pool = b * blocks + b * blocks // 4 + 3
    table = torch.randperm(pool, generator=g)[: b * blocks].view(b, blocks).int().cuda()
    k, v = _kv(case, blocks * BLOCK, seed * 7 + 3)
    records = _records(kind, k, v)
    arena = torch.zeros((pool, h, records.shape[-1]), dtype=torch.uint8, device="cuda")
    arena[table.long()] = records
    del records
    residual = None
    if kind != "bf16":
        first = (stored // GROUP * GROUP).cuda().clamp_max(blocks * BLOCK - GROUP)
        rows = first[:, None] + torch.arange(GROUP, device="cuda")
        residual = k[torch.arange(b, device="cuda")[:, None], rows].transpose(1, 2).contiguous()  # [B, H, 32, D]
    return {"arena": arena, "table": table, "residual": residual}


def _handle(case, s):
    """The framework's handle of the cell (the program that serves keeps it from call to call)."""
    import mixed_precision_kv_loopkv_b200 as kvlib
    cell = case["op"] != "norm_rope"
    kv = kvlib.KVCells([case["kind"] if cell else "bf16"], 1, 1, case["heads"], case["dim"],
                       s["arena"].shape[0] if cell else 1, case["batch"], s["table"].shape[1] if cell else 1,
                       num_kv_heads=case["kv_heads"])
    if cell:
        kv.arena_view(0).copy_(s["arena"])
        if s["residual"] is not None:
            kv.residuals[0].copy_(s["residual"])
    rotary = None
    if case["op"] in ("norm_rope", "append"):
        rotary = kvlib.Rotary(s["cos_sin"], interleaved=case["pairs"] == "neighbours", q_weight=s["q_weight"],
                              k_weight=s["k_weight"], eps=EPS)
    return kvlib, kv, rotary


def prepare(case, seed):
    b, t, h, hk, d = (case[x] for x in ("batch", "tokens", "heads", "kv_heads", "dim"))
    before, new = _lengths(case, seed)
    total = before + new
    s = {"case": case, "start": before.int().cuda(), "new": new.int().cuda() if case["ragged"] else None}
    if case["op"] in ("norm_rope", "append"):
        qkv = _random((b, t, (h + 2 * hk) * d), seed * 7 + 4).bfloat16()     # one projection's output; q, k, v are views
        s["q"], s["k"], s["v"] = (x.unflatten(-1, (-1, d)) for x in qkv.split([h * d, hk * d, hk * d], -1))
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = torch.arange(int(total.max()), device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_weight"] = (1 + _random((d,), seed * 7 + 5, 0.2)).bfloat16() if case["norm"] else None
        s["k_weight"] = (1 + _random((d,), seed * 7 + 6, 0.2)).bfloat16() if case["norm"] else None
        s["q_out"] = torch.zeros((b, t, h, d), dtype=torch.bfloat16, device="cuda")
    if case["op"] == "norm_rope":
        s["k_out"] = torch.zeros((b, t, hk, d), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "append":
        s.update(_cell(case, before, int(total.max()), seed))
        slots = -(-(t + GROUP - 1) // GROUP) * GROUP
        s["first"], s["end"], s["slots"] = (before // GROUP * GROUP).int().cuda(), total.int().cuda(), slots
        s["k_out"], s["v_out"] = (torch.zeros((b, slots, hk, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    elif case["op"] == "read":
        # the last tokens of what is stored; a sequence with fewer leaves the rest of its rows as they are
        stored = torch.maximum(before, new)
        s.update(_cell(case, stored, int(stored.max()), seed))
        s["first"], s["end"] = (stored - new).int().cuda(), stored.int().cuda()
        s["k_out"], s["v_out"] = (torch.zeros((b, t, hk, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    elif case["op"] == "chunk":
        stored = total if case["mode"] == "stored" else before
        s.update(_cell(case, stored, max(1, int(stored.max())), seed))
        s["stored"], s["longest"] = stored.int().cuda(), int(stored.max())
        s["q"] = _random((b, t, h, d), seed * 7 + 8, 0.125).bfloat16()
        s["out"] = torch.zeros_like(s["q"])
        if case["mode"] == "current":
            s["k_cur"], s["v_cur"] = _kv(case, t, seed * 7 + 9)
    if own:
        s["handle"] = _handle(case, s)
    return s


# ------------------------------------------------------------- plain forms


def _valid(s):
    """Which of the chunk's rows are there, [B, T, 1, 1]."""
    t = s["case"]["tokens"]
    new = s["new"] if s["new"] is not None else torch.full_like(s["start"], t)
    return (torch.arange(t, device="cuda") < new[:, None])[:, :, None, None]


def _norm_rope(s, x, weight):
    """fp32 result, before the rounding to bf16 (rows [B, T, heads, D])."""
    case, x = s["case"], x.float()
    if weight is not None:
        r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + EPS).float()
        x = (x * r) * weight.float()
    rot, half = case["rot"], case["rot"] // 2
    pos = (s["start"][:, None] + torch.arange(x.shape[1], device="cuda")).clamp_max(s["cos_sin"].shape[0] - 1)
    cos, sin = s["cos_sin"][pos][:, :, None].split(half, -1)
    if case["pairs"] == "halves":
        a, c = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - c * sin, c * cos + a * sin], -1)
    else:
        a, c = x[..., :rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _codes(row_bytes):
    """Bytes [..., n] -> 2-bit codes uint8 [..., 4 n]."""
    shifts = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device="cuda")
    return ((row_bytes[..., None] >> shifts) & 3).flatten(-2)


def _stored(s, table, open_from):
    """fp32 keys and values [B, Hkv, S, D] of the blocks in `table` [B, S / 16]; keys of the tokens from
    open_from[b] on come from the exact rows of the open group."""
    case, d = s["case"], s["case"]["dim"]
    rec = s["arena"][table.long()].transpose(1, 2)                                     # [B, H, n, record]
    meta = lambda x: x.contiguous().view(torch.bfloat16).float().unflatten(-1, (-1, 2))  # noqa: E731
    if case["kind"] == "bf16":
        k, v = (x.contiguous().view(torch.bfloat16).float().unflatten(-1, (BLOCK, d)).flatten(2, 3)
                for x in rec.split(BLOCK * d * 2, -1))
        return k, v
    plane, km, vm = BLOCK * d // 4, d * 2, BLOCK * (d // GROUP) * 4
    rows = lambda x: _codes(x.unflatten(-1, (BLOCK, d // 4)))                           # noqa: E731
    columns = lambda x: _codes(x.unflatten(-1, (d // 4, BLOCK)).transpose(-1, -2))      # noqa: E731
    if case["kind"] == "q4":
        k_hi, k_lo, k_meta, v_hi, v_meta, v_lo = rec.split([plane, plane, km, plane, vm, plane], -1)
        kc, vc = (rows(k_hi) << 2) | rows(k_lo), (columns(v_hi) << 2) | rows(v_lo)
    else:
        k_hi, k_meta, v_hi, v_meta = rec.split([plane, km, plane, vm], -1)
        kc, vc = rows(k_hi), columns(v_hi)
    k_meta = meta(k_meta).unflatten(2, (-1, 2)).flatten(3, 4)                           # [B, H, groups, D, 2]
    kc = kc.flatten(2, 3).unflatten(2, (-1, GROUP))
    k = torch.addcmul(k_meta[:, :, :, None, :, 1], k_meta[:, :, :, None, :, 0], kc.float()).flatten(2, 3)
    v_meta = meta(v_meta).unflatten(-2, (BLOCK, d // GROUP))[..., None, :]              # [B, H, n, 16, D / 32, 1, 2]
    v = torch.addcmul(v_meta[..., 1], v_meta[..., 0], vc.unflatten(-1, (-1, GROUP)).float()).flatten(-2).flatten(2, 3)
    at = torch.arange(k.shape[2], device="cuda")
    opened = s["residual"].float()[:, :, at % GROUP]
    return torch.where((at >= open_from[:, None])[:, None, :, None], opened, k), v


def _append(s):
    """Rotated queries, and the cell's tokens from the start of the first group that the chunk touches."""
    case, slots = s["case"], s["slots"]
    there = _valid(s)
    q = torch.where(there, _norm_rope(s, s["q"], s["q_weight"]), 0).bfloat16()
    k_new = _norm_rope(s, s["k"], s["k_weight"]).bfloat16().float()
    v_new = s["v"].float()
    at = torch.arange(slots, device="cuda")
    i = at - (s["start"] - s["first"])[:, None]                                         # slot -> row of the chunk
    row = i.clamp(0, case["tokens"] - 1).long()
    seq = torch.arange(case["batch"], device="cuda")[:, None]
    # what the open group held before
    n = s["table"].shape[1]
    blocks = torch.gather(s["table"], 1, ((s["first"] // BLOCK)[:, None] + torch.arange(2, device="cuda")).clamp_max(n - 1).long())
    k_old, v_old = (x.transpose(1, 2)[:, at % GROUP] for x in _stored(s, blocks, torch.zeros_like(s["first"])))
    old = (i < 0)[..., None, None]
    k, v = torch.where(old, k_old, k_new[seq, row]), v_new[seq, row]
    if case["kind"] != "bf16":
        bits = BITS[case["kind"]]
        code, scale, low = _quantise(k.unflatten(1, (-1, GROUP)), bits, 2)
        full = at // GROUP * GROUP + GROUP <= (s["end"] - s["first"])[:, None]
        k = torch.where(full[..., None, None], torch.addcmul(low, scale, code).flatten(1, 2), k)
        code, scale, low = _quantise(v.unflatten(3, (-1, GROUP)), bits, 4)
        v = torch.addcmul(low, scale, code).flatten(3, 4)
    v = torch.where(old, v_old, v)
    kept = (at < (s["end"] - s["first"])[:, None])[..., None, None]
    return q, torch.where(kept, k, 0).bfloat16(), torch.where(kept, v, 0).bfloat16()


def _read(s):
    k, v = (x.transpose(1, 2) for x in _stored(s, s["table"], s["end"] // GROUP * GROUP))
    t = s["case"]["tokens"]
    pos = s["first"][:, None] + torch.arange(t, device="cuda")
    kept = (pos < s["end"][:, None])[..., None, None]
    seq, pos = torch.arange(s["case"]["batch"], device="cuda")[:, None], pos.clamp_max(k.shape[1] - 1).long()
    return torch.where(kept, k[seq, pos], 0).bfloat16(), torch.where(kept, v[seq, pos], 0).bfloat16()


def _chunk(s):
    case = s["case"]
    b, t, h, hk, d = (case[x] for x in ("batch", "tokens", "heads", "kv_heads", "dim"))
    k, v = _stored(s, s["table"], s["stored"] // GROUP * GROUP)                          # [B, Hkv, S, D]
    at = torch.arange(k.shape[2], device="cuda")
    i = torch.arange(t, device="cuda")
    seen = at < s["stored"][:, None, None]                                              # [B, 1, S]
    if case["mode"] == "stored":
        seen = seen & (at <= s["start"][:, None, None] + i[:, None])
    else:
        seen = torch.cat([seen.expand(b, t, -1), (i <= i[:, None]).expand(b, t, t)], -1)
        k = torch.cat([k, s["k_cur"].float().transpose(1, 2)], 2)
        v = torch.cat([v, s["v_cur"].float().transpose(1, 2)], 2)
    v = torch.where(seen.any(1)[:, None, :, None], v, 0)
    q = s["q"].float().unflatten(2, (hk, h // hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G T, D]
    logit = (q @ k.transpose(2, 3)).unflatten(2, (-1, t))
    logit.masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(logit - logit.amax(-1, keepdim=True))
    out = (p / p.sum(-1, keepdim=True)).flatten(2, 3) @ v
    out = out.unflatten(2, (-1, t)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return torch.where(_valid(s), out, 0).bfloat16()


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        kvlib, kv, rotary = s["handle"]
        if op == "norm_rope":
            return kvlib.loopkv_norm_rope(rotary, s["q"], s["k"], s["start"], new_lens=s["new"], q_out=s["q_out"], k_out=s["k_out"])
        if op == "append":
            kvlib.loopkv_rope_append(kv, 0, 0, rotary, s["q"], s["k"], s["v"], s["table"], s["start"], new_lens=s["new"],
                                     q_out=s["q_out"])
            return s["q_out"], *kvlib.loopkv_read_tokens(kv, 0, 0, s["table"], s["end"], s["first"], s["slots"],
                                                         k_out=s["k_out"], v_out=s["v_out"])
        if op == "read":
            return kvlib.loopkv_read_tokens(kv, 0, 0, s["table"], s["end"], s["first"], s["case"]["tokens"],
                                            k_out=s["k_out"], v_out=s["v_out"])
        return kvlib.loopkv_chunk_attention(kv, 0, 0, s["q"], s["table"], s["start"], new_lens=s["new"], sm_scale=1.0, out=s["out"],
                                            max_seq_len=s["longest"], k_cur=s.get("k_cur"), v_cur=s.get("v_cur"))
    if op == "norm_rope":
        there = _valid(s)
        return tuple(torch.where(there, _norm_rope(s, s[x], s[x + "_weight"]), 0).bfloat16() for x in "qk")
    return {"append": _append, "read": _read, "chunk": _chunk}[op](s)


def work(case):
    """Bytes and operations of one pass.  Ragged lengths count as what _lengths gives for seed 0."""
    before, new = _lengths(case, 0)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    kind, n = case.get("kind"), int(new.sum())
    token = {"q4": d + d // 8 * 2, "q2": d // 2 + d // 8 * 2, "bf16": 4 * d}.get(kind, 0) * hk   # stored bytes of one token
    if case["op"] == "norm_rope":
        return {"bytes": n * (h + hk) * d * 4, "flops": n * (h + hk) * d * 7}
    if case["op"] == "append":
        back = int((before + new - before // GROUP * GROUP).sum())
        return {"bytes": n * (h * d * 4 + hk * d * 4 + token) + back * hk * d * 4, "flops": n * (h + 2 * hk) * d * 8}
    if case["op"] == "read":
        return {"bytes": n * (token + hk * d * 4), "flops": n * hk * d * 4}
    stored = before + new if case["mode"] == "stored" else before
    pairs = int((new * before + new * (new + 1) // 2).sum())
    fresh = 0 if case["mode"] == "stored" else n * hk * d * 4
    return {"bytes": int(stored.sum()) * token + fresh + n * h * d * 4, "flops": 4 * pairs * h * d}


# ------------------------------------------------------ 64 bits, head by head


def _exact_turn(case, s, x, weight, b, n):
    """Rows x[b, :n] normed and rotated: each pair as one complex number."""
    x = x[b, :n].double()
    if weight is not None:
        x = x / (x.square().sum(-1, keepdim=True) / case["dim"] + EPS).sqrt() * weight.double()
    rot, half = case["rot"], case["rot"] // 2
    p = int(s["start"][b])
    table = s["cos_sin"][p: p + n].double()
    turn = torch.complex(table[:, :half], table[:, half:])[:, None]
    y = x.clone()
    first = slice(0, half) if case["pairs"] == "halves" else slice(0, rot, 2)
    second = slice(half, rot) if case["pairs"] == "halves" else slice(1, rot, 2)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_bits(data, width):
    """uint8 [..., n] -> the 4 n two-bit codes, as 64-bit floats."""
    wide = data.long()
    out = torch.empty(*data.shape, 4, dtype=torch.float64, device="cuda")
    for j in range(4):
        out[..., j] = (wide // 4**j) % 4
    return out.reshape(*data.shape[:-1], width)


def _exact_cell(case, s, b, h, n):
    """The n stored tokens' keys and values of one sequence and head, block after block of the table."""
    d, kind = case["dim"], case["kind"]
    blocks = -(-n // GROUP) * 2
    rec = s["arena"][s["table"][b, :blocks].long(), h]
    if kind == "bf16":
        both = rec.view(torch.bfloat16).double().view(blocks, 2, BLOCK, d)
        return both[:, 0].reshape(-1, d)[:n], both[:, 1].reshape(-1, d)[:n]
    q4, pl = kind == "q4", BLOCK * d // 4
    at, part = 0, {}
    for name, size in (("kh", pl), ("kl", pl if q4 else 0), ("km", 2 * d), ("vh", pl), ("vm", d // 2 * 4), ("vl", pl if q4 else 0)):
        part[name] = rec[:, at: at + size]
        at += size
    num = lambda x, *shape: x.contiguous().view(torch.bfloat16).double().view(*shape)  # noqa: E731
    kc = _exact_bits(part["kh"].reshape(blocks * BLOCK, -1), d)
    vc = _exact_bits(part["vh"].reshape(blocks, d // 4, BLOCK).transpose(1, 2).reshape(blocks * BLOCK, -1), d)
    if q4:
        kc = 4 * kc + _exact_bits(part["kl"].reshape(blocks * BLOCK, -1), d)
        vc = 4 * vc + _exact_bits(part["vl"].reshape(blocks * BLOCK, -1), d)
    km = num(part["km"], blocks // 2, d, 2).repeat_interleave(GROUP, 0)
    vm = num(part["vm"], blocks * BLOCK, d // GROUP, 2).repeat_interleave(GROUP, 1)
    k, v = (km[..., 1] + km[..., 0] * kc)[:n], (vm[..., 1] + vm[..., 0] * vc)[:n]
    if n % GROUP:
        k[n // GROUP * GROUP:] = s["residual"][b, h, : n % GROUP].double()
    return k, v


def _exact_groups(x, bits):
    """x fp64 [groups, members, rest] quantised over its members and back."""
    low, high = x.amin(1, keepdim=True), x.amax(1, keepdim=True)
    scale = ((high - low) / (2**bits - 1)).float().bfloat16().double()
    steps = torch.where(scale == 0, 0.0, (x - low) / torch.where(scale == 0, 1.0, scale))
    return low + scale * torch.round(steps).clamp(0, 2**bits - 1)


def exact(case, seed):
    s = prepare(case, seed)
    b, t, h, hk, d = (case[x] for x in ("batch", "tokens", "heads", "kv_heads", "dim"))
    start = s["start"].tolist()
    new = s["new"].tolist() if s["new"] is not None else [t] * b
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if case["op"] == "norm_rope":
        out = zeros(b, t, h, d), zeros(b, t, hk, d)
        for i in range(b):
            for o, x, w in zip(out, (s["q"], s["k"]), (s["q_weight"], s["k_weight"])):
                o[i, : new[i]] = _exact_turn(case, s, x, w, i, new[i])
        return out
    if case["op"] == "read":
        k_out, v_out = zeros(b, t, hk, d), zeros(b, t, hk, d)
        for i in range(b):
            for j in range(hk):
                k, v = _exact_cell(case, s, i, j, int(s["end"][i]))
                n = min(t, k.shape[0] - int(s["first"][i]))
                k_out[i, :n, j], v_out[i, :n, j] = k[int(s["first"][i]):][:n], v[int(s["first"][i]):][:n]
        return k_out, v_out
    if case["op"] == "append":
        q_out, k_out, v_out = zeros(b, t, h, d), zeros(b, s["slots"], hk, d), zeros(b, s["slots"], hk, d)
        for i in range(b):
            q_out[i, : new[i]] = _exact_turn(case, s, s["q"], s["q_weight"], i, new[i])
            fresh = _exact_turn(case, s, s["k"], s["k_weight"], i, new[i]).float().bfloat16().double()
            had, lo = start[i], int(s["first"][i])
            k = zeros(had - lo + new[i], hk, d)
            v = zeros(had - lo + new[i], hk, d)
            for j in range(hk):
                if had > lo:
                    old_k, old_v = _exact_cell(case, s, i, j, had)
                    k[: had - lo, j], v[: had - lo, j] = old_k[lo:], old_v[lo:]
            k[had - lo:], v[had - lo:] = fresh, s["v"][i, : new[i]].double()
            if case["kind"] != "bf16":
                bits, whole = BITS[case["kind"]], k.shape[0] // GROUP * GROUP
                if whole:
                    k[:whole] = _exact_groups(k[:whole].reshape(-1, GROUP, hk * d), bits).reshape(whole, hk, d)
                v[had - lo:] = _exact_groups(v[had - lo:].reshape(-1, GROUP, 1), bits).reshape(new[i], hk, d)
            k_out[i, : k.shape[0]], v_out[i, : v.shape[0]] = k, v
        return q_out, k_out, v_out
    out = zeros(b, t, h, d)
    for i in range(b):
        n = int(s["stored"][i])
        rows = torch.arange(new[i], device="cuda")[:, None]
        for j in range(hk):
            k, v = _exact_cell(case, s, i, j, n)
            last = start[i] + rows                                   # the last key that each row sees
            if case["mode"] == "current":
                k, v = torch.cat([k, s["k_cur"][i, : new[i], j].double()]), torch.cat([v, s["v_cur"][i, : new[i], j].double()])
            hidden = torch.arange(k.shape[0], device="cuda") > last
            for g in range(h // hk):
                head = j * (h // hk) + g
                x = (s["q"][i, : new[i], head].double() @ k.T).masked_fill_(hidden, -math.inf)
                out[i, : new[i], head] = torch.softmax(x, -1) @ v
    return out
