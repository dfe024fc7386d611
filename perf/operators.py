"""The sparse decode operators next to the residency path, and how they are timed.

Three operators on one cache of 656-byte Q8G64 rows and 128-value index keys,
held in blocks that a table maps (or one contiguous run per sequence):

``append``  a token's latent, position part and index key become a cache row:
            the position part rotated by the token's position, the latent
            quantised to int8 in groups of 64, the key to e4m3 or bf16.
``score``   the cheap score that the top-k selection reads:
            scale_j * sum_h w_h * max(0, q_h . key_j) for every cached
            position, or its maximum over each block of positions.
``attend``  softmax attention of absorbed MLA queries over the rows of the
            selected positions or blocks, or over all rows of a sequence.

``run`` computes them in elementary torch operations, or with the library's
calls where ``own`` is set.
"""
import math

import torch

own = False

ROW, LATENT, ROPE, GROUPS, KEY = 656, 512, 64, 8, 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
THETA = 10_000.0
E4M3_MAX = 448.0

_handle = None


def listed():
    return [
        # one token of one stream: what every decode step of every layer pays
        dict(name="append_one_token", op="append", seqs=1, tokens=1, first=50_022, dtype="bf16", interleaved=True,
             key="e4m3", block_rows=16),
        # a decode step of a batch far into long contexts, half-split pairs, keys kept in bf16
        dict(name="append_batch_far", op="append", seqs=61, tokens=61, first=1_048_500, dtype="fp16",
             interleaved=False, key="bf16", block_rows=16),
        # the prefill of one 60,000-token session into its pool blocks
        dict(name="append_prefill_60k", op="append", seqs=1, tokens=60_000, first=0, dtype="bf16", interleaved=True,
             key="e4m3", block_rows=16),
        # ragged prefill pieces of several sessions from an fp32 projection
        dict(name="append_ragged_fp32", op="append", seqs=7, tokens=16_381, first=1_003, dtype="fp32",
             interleaved=True, key="e4m3", block_rows=64),
        # the selection scores of one decode step over a 50K context
        dict(name="score_50k", op="score", seqs=1, per_seq=1, heads=64, length=50_023, ragged=False, dtype="e4m3",
             block=1, block_rows=0),
        # a verification round: four draft positions of one stream, keys in bf16
        dict(name="score_mtp4", op="score", seqs=1, per_seq=4, heads=64, length=50_027, ragged=False, dtype="bf16",
             block=1, block_rows=0),
        # block scores of a million-token context in pool blocks
        dict(name="score_1m_blocks", op="score", seqs=1, per_seq=1, heads=64, length=1_048_576, ragged=False,
             dtype="e4m3", block=16, block_rows=16),
        # a batch of uneven contexts, an empty one among them, an odd number of heads
        dict(name="score_batch_ragged", op="score", seqs=13, per_seq=2, heads=24, length=20_011, ragged=True,
             dtype="e4m3", block=1, block_rows=16),
        # the 2,048 gathered rows of one layer's decode step (the output of the resolve/gather)
        dict(name="attend_gathered", op="attend", seqs=1, per_seq=1, heads=64, length=2_048, ragged=False, picked=0,
             sel_block=1, block_rows=0),
        # a served batch, every stream with its own 2,048 positions in the pool
        dict(name="attend_batch_positions", op="attend", seqs=64, per_seq=1, heads=64, length=16_384, ragged=False,
             picked=2_048, sel_block=1, block_rows=16),
        # whole blocks selected, uneven contexts, an empty one, an odd head count, two draft positions
        dict(name="attend_blocks_ragged", op="attend", seqs=9, per_seq=2, heads=20, length=12_345, ragged=True,
             picked=61, sel_block=16, block_rows=16),
        # one stream over everything it has: a million rows and 128 heads
        dict(name="attend_dense_1m", op="attend", seqs=1, per_seq=1, heads=128, length=1_048_576, ragged=False,
             picked=0, sel_block=1, block_rows=16),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "score", "attend"])
    if op == "append":
        tokens = _spread(rng, 1, 60_000)
        # a decode step has one token a sequence, a prefill has runs
        seqs = tokens if tokens <= 256 and rng.random() < 0.5 else rng.randint(1, min(tokens, 16))
        return dict(op=op, seqs=seqs, tokens=tokens, first=_spread(rng, 1, 1_048_576) - 1,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), interleaved=rng.random() < 0.5,
                    key=rng.choice(["none", "bf16", "e4m3"]), block_rows=rng.choice([4, 16, 48, 64]))
    if op == "score":
        seqs, per_seq = _spread(rng, 1, 32), rng.choice([1, 1, 2, 4])
        return dict(op=op, seqs=seqs, per_seq=per_seq, heads=rng.choice([1, 8, 16, 24, 32, 64]),
                    length=_spread(rng, 1, 1_048_576 // (seqs * per_seq)), ragged=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "e4m3"]), block=rng.choice([1, 1, 16, 64]),
                    block_rows=rng.choice([0, 16, 48, 64]))
    seqs, per_seq, heads = _spread(rng, 1, 128), rng.choice([1, 1, 2, 4]), rng.choice([1, 8, 16, 20, 64, 128])
    budget = max(64, 524_288 // (seqs * per_seq))
    sel_block = rng.choice([0, 1, 1, 16, 64])
    if sel_block == 0:  # every row of the sequence
        return dict(op=op, seqs=seqs, per_seq=per_seq, heads=heads, length=_spread(rng, 1, budget),
                    ragged=rng.random() < 0.5, picked=0, sel_block=1, block_rows=rng.choice([0, 16, 48]))
    picked = _spread(rng, 1, max(1, min(4_096, budget) // sel_block))
    length = _spread(rng, picked * sel_block, max(picked * sel_block, 2_000_000 // seqs))
    return dict(op=op, seqs=seqs, per_seq=per_seq, heads=heads, length=length, ragged=rng.random() < 0.5,
                picked=picked, sel_block=sel_block, block_rows=rng.choice([0, 16, 48]))


# ------------------------------------------------------------------ sizes
def _lengths(case):
    """Each query's visible positions, [sequences][queries of a sequence]."""
    s_n, q_n, n = case["seqs"], case["per_seq"], case["length"]
    out = []
    for s in range(s_n):
        have = n - (n * ((s * 37) % 64)) // 96 - (s % 5) if case["ragged"] else n
        if case["ragged"] and s_n > 2 and s == s_n - 1:
            have = 0
        out.append([max(0, have - (q_n - 1 - i)) for i in range(q_n)])
    return out


def _tokens(case):
    """(sequence, position) of every appended token: runs of a sequence's next positions."""
    n, s_n = case["tokens"], case["seqs"]
    seq = torch.arange(n, dtype=torch.int64) * s_n // n
    start = torch.searchsorted(seq, torch.arange(s_n))
    return seq, case["first"] + torch.arange(n) - start[seq] + (seq * 3) % 7


def work(case):
    if case["op"] == "append":
        n, size = case["tokens"], torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
        key = {"none": 0, "bf16": KEY * (size + 2), "e4m3": KEY * (size + 1) + 4}[case["key"]]
        # inputs, row, dequantised copy, key, sequence and position; two operations a value to scale and round
        return dict(bytes=n * ((LATENT + ROPE) * size + ROW + 2 * (LATENT + ROPE) + key + 8),
                    flops=n * (4 * LATENT + 6 * ROPE))
    lens = _lengths(case)
    seen = sum(map(sum, lens))
    held = sum(map(max, lens))
    nq, heads = case["seqs"] * case["per_seq"], case["heads"]
    if case["op"] == "score":
        size = 2 if case["dtype"] == "bf16" else 1
        row = KEY * size + (4 if size == 1 else 0)
        return dict(bytes=held * row + nq * heads * (KEY * size + 4) + 4 * nq * -(-case["length"] // case["block"]),
                    flops=seen * heads * (2 * KEY + 3))
    units, block = case["picked"], case["sel_block"]
    read = [[min(n, units * block) if units else n for n in row] for row in lens]
    rows = sum(min(max(have), sum(r)) if units else max(have) for have, r in zip(lens, read))
    return dict(bytes=rows * ROW + 4 * nq * units + nq * heads * (2 * (LATENT + ROPE) + 2 * LATENT + 4),
                flops=sum(map(sum, read)) * heads * (2 * (LATENT + ROPE) + 2 * LATENT + 4))


# ----------------------------------------------------------------- inputs
def _inv_freq():
    return THETA ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)


def _table(case, blocks, g):
    """A shuffled block table and the number of blocks behind it."""
    spare = 3
    total = case["seqs"] * blocks + spare
    ids = torch.randperm(total, generator=g, device="cuda")[:case["seqs"] * blocks]
    return ids.view(case["seqs"], blocks).to(torch.int32), total


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"
    state = dict(case=case)
    if case["op"] == "append":
        n, dt = case["tokens"], DTYPES[case["dtype"]]
        seq, pos = _tokens(case)
        # one projection's output: latent and position part side by side, some channels much larger than others
        gain = torch.exp(torch.randn(LATENT + ROPE, generator=g, device=dev))
        kv = (torch.randn(n, LATENT + ROPE, generator=g, device=dev) * gain).to(dt)
        br = case["block_rows"]
        first = int(pos.min()) // br                      # earlier blocks of a sequence are not in the table's window
        blocks = int(pos.max()) // br - first + 1
        table, total = _table(case, blocks, g)
        if first:                                         # positions count from the sequence's first token
            table = torch.cat([torch.full((case["seqs"], first), -1, dtype=torch.int32, device=dev), table], 1)
        state.update(kv=kv, seq=seq.to(torch.int32).to(dev), pos=pos.to(torch.int32).to(dev), table=table,
                     block_rows=br, inv_freq=_inv_freq(),
                     rows=torch.zeros(total * br, ROW, dtype=torch.uint8, device=dev),
                     values=torch.empty(n, LATENT + ROPE, dtype=torch.bfloat16, device=dev))
        if case["key"] != "none":
            state["key"] = (torch.randn(n, KEY, generator=g, device=dev) * gain[:KEY]).to(dt)
            state["keys"] = torch.zeros(total * br, KEY, dtype=torch.bfloat16, device=dev)
            if case["key"] == "e4m3":
                state["keys"] = torch.zeros(total * br, KEY, dtype=torch.uint8, device=dev).view(DTYPES["e4m3"])
                state["key_scales"] = torch.zeros(total * br, dtype=torch.float32, device=dev)
        return state

    s_n, nq, heads, n = case["seqs"], case["seqs"] * case["per_seq"], case["heads"], case["length"]
    br = case["block_rows"] or n
    if case["block_rows"]:
        state["table"], total = _table(case, -(-n // br), g)
    else:
        state["table"], total = None, s_n
    state["block_rows"] = br
    state["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev).view(nq)
    if case["op"] == "score":
        dt = DTYPES[case["dtype"]]
        state["q"] = torch.randn(nq, heads, KEY, generator=g, device=dev).to(dt)
        state["w"] = torch.randn(nq, heads, generator=g, device=dev) / math.sqrt(heads * KEY)
        state["keys"] = torch.randn(total * br, KEY, generator=g, device=dev).to(dt)
        if case["dtype"] == "e4m3":
            state["key_scales"] = torch.exp2(torch.randint(-6, 1, (total * br,), generator=g, device=dev).float())
        state["out"] = torch.empty(nq, -(-n // case["block"]), dtype=torch.float32, device=dev)
        return state

    rows = torch.empty(total * br, ROW, dtype=torch.uint8, device=dev)
    rows.view(torch.int8)[:, :LATENT] = torch.randint(-127, 128, (total * br, LATENT), generator=g, device=dev,
                                                      dtype=torch.int8)
    rows.view(torch.float16)[:, LATENT // 2:LATENT // 2 + GROUPS] = (
        torch.rand(total * br, GROUPS, generator=g, device=dev) * 9e-3 + 1e-3).half()
    rows.view(torch.bfloat16)[:, LATENT // 2 + GROUPS:] = torch.randn(total * br, ROPE, generator=g,
                                                                     device=dev).bfloat16()
    state["rows"] = rows
    state["q"] = torch.randn(nq, heads, LATENT + ROPE, generator=g, device=dev).bfloat16()
    state["scale"] = 192 ** -0.5
    state["sel"] = None
    if case["picked"]:
        # what the top-k selection returns: the units with the best scores, ascending; those past a short
        # sequence's end only where it has too few
        units = -(-n // case["sel_block"])
        score = torch.rand(nq, units, generator=g, device=dev)
        start = torch.arange(units, device=dev) * case["sel_block"]
        score.masked_fill_(start[None, :] >= state["lens"][:, None], -math.inf)
        state["sel"] = score.topk(case["picked"], dim=1).indices.sort(dim=1).values.to(torch.int32)
    state["out"] = torch.empty(nq, heads, LATENT, dtype=torch.bfloat16, device=dev)
    state["lse"] = torch.empty(nq, heads, dtype=torch.float32, device=dev)
    return state


# -------------------------------------------------------------- plain form
def _places(table, block_rows, seq, pos):
    """The cache row of each sequence's position (broadcast over both)."""
    if table is None:
        return seq * block_rows + pos
    return table[seq, pos // block_rows].long() * block_rows + pos % block_rows


def _values_of_rows(rows):
    """What rows stand for, as the cache's dequantised rows have it: bf16 of int8 * scale, and the position part."""
    q = rows[..., :LATENT].contiguous().view(torch.int8).float()
    scale = rows[..., LATENT:LATENT + 2 * GROUPS].contiguous().view(torch.float16).float()
    latent = (q.unflatten(-1, (GROUPS, 64)) * scale[..., None]).flatten(-2).bfloat16()
    return latent.float(), rows[..., LATENT + 2 * GROUPS:].contiguous().view(torch.bfloat16).float()


def _scale_up(amax):
    """The smallest fp16 with 127 * scale >= amax (a NaN where amax is not finite)."""
    near = (amax.double() / 127).clamp(max=65504.0)
    h = near.to(torch.float16)
    bits = h.view(torch.int16)
    bits = torch.where(h.double() < near, bits + 1, bits)
    return torch.where(amax.isfinite(), bits.view(torch.float16), torch.tensor(math.nan, device=amax.device).half())


def _append(st):
    case = st["case"]
    latent, rope = st["kv"][:, :LATENT].float(), st["kv"][:, LATENT:].float()
    seq, pos = st["seq"].long(), st["pos"].long()
    at = _places(st["table"], st["block_rows"], seq, pos)
    grouped = latent.unflatten(1, (GROUPS, 64))
    scale = _scale_up(grouped.abs().amax(2))
    q = (grouped.double() / scale.double()[..., None]).round().nan_to_num(0.0).clamp(-127, 127)
    q = torch.where(scale[..., None] > 0, q, torch.zeros_like(q)).to(torch.int8)
    angle = pos.double()[:, None] * st["inv_freq"].to(pos.device)
    c, s = angle.cos().float(), angle.sin().float()
    if case["interleaved"]:
        a, b = rope[:, 0::2], rope[:, 1::2]
        turned = torch.stack([a * c - b * s, b * c + a * s], 2).flatten(1)
    else:
        a, b = rope[:, :ROPE // 2], rope[:, ROPE // 2:]
        turned = torch.cat([a * c - b * s, b * c + a * s], 1)
    turned = turned.bfloat16()
    rows = st["rows"]
    rows[at] = torch.cat([q.flatten(1).view(torch.uint8), scale.view(torch.uint8), turned.view(torch.uint8)], 1)
    values = torch.cat([(q.float() * scale.float()[..., None]).flatten(1).bfloat16(), turned], 1)
    if case["key"] == "bf16":
        st["keys"][at] = st["key"].bfloat16()
    elif case["key"] == "e4m3":
        amax = st["key"].float().abs().amax(1)
        part, power = torch.frexp(amax.double() / E4M3_MAX)   # the smallest power of two at or above amax / 448
        step = torch.exp2((power - (part == 0.5).to(power.dtype)).float()).clamp(min=2.0 ** -100)
        st["keys"].view(torch.uint8)[at] = (st["key"].float() / step[:, None]).to(DTYPES["e4m3"]).view(torch.uint8)
        st["key_scales"][at] = step
    return _appended(st, values)


def _appended(st, values):
    rows = st["rows"]
    out = [values, rows.view(torch.int8)[:, :LATENT],
           rows.view(torch.float16)[:, LATENT // 2:LATENT // 2 + GROUPS],
           rows.view(torch.bfloat16)[:, LATENT // 2 + GROUPS:]]
    out += [st[k] for k in ("keys", "key_scales") if k in st]
    return out


def _score(st):
    case = st["case"]
    s_n, q_n, heads, n, block = case["seqs"], case["per_seq"], case["heads"], case["length"], case["block"]
    pos = torch.arange(n, device="cuda")
    at = _places(st["table"], st["block_rows"], torch.arange(s_n, device="cuda")[:, None], pos)
    keys = (st["keys"].view(torch.uint8)[at].view(DTYPES["e4m3"]) if case["dtype"] == "e4m3"
            else st["keys"][at]).float()
    q = st["q"].float().view(s_n, q_n * heads, KEY)
    dots = torch.relu(q @ keys.transpose(1, 2)).view(s_n, q_n, heads, n)
    total = (dots * st["w"].view(s_n, q_n, heads, 1)).sum(2)
    if case["dtype"] == "e4m3":
        total = total * st["key_scales"][at][:, None]
    total = total.masked_fill(pos >= st["lens"].view(s_n, q_n, 1), -math.inf).view(s_n * q_n, n)
    if block == 1:
        return total
    wide = torch.nn.functional.pad(total, (0, -n % block), value=-math.inf)
    return wide.unflatten(1, (-1, block)).amax(2)


def _attend(st):
    case = st["case"]
    nq, q_n, n = st["q"].shape[0], case["per_seq"], case["length"]
    lens = st["lens"].long()
    seq = torch.arange(nq, device="cuda") // q_n
    if st["sel"] is None:
        pos = torch.arange(n, device="cuda").expand(nq, n)
    else:
        b = case["sel_block"]
        pos = (st["sel"].long()[..., None] * b + torch.arange(b, device="cuda")).flatten(1)
    valid = (pos >= 0) & (pos < lens[:, None])
    at = _places(st["table"], st["block_rows"], seq[:, None], torch.where(valid, pos, 0))
    latent, rope = _values_of_rows(st["rows"][at])
    q = st["q"].float()
    logits = (q[..., :LATENT] @ latent.transpose(1, 2) + q[..., LATENT:] @ rope.transpose(1, 2)) * st["scale"]
    logits = logits.masked_fill(~valid[:, None], -math.inf)
    top = logits.amax(2, keepdim=True)
    p = torch.exp(logits - torch.where(top.isfinite(), top, 0.0))
    total = p.sum(2, keepdim=True)
    out = (p @ latent) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + torch.where(top.isfinite(), top, 0.0)
    return out.bfloat16(), lse[..., 0]


# ---------------------------------------------------------- the library's calls
def _open(st):
    """The context (one for all) and the view of this state's cache, kept as a program keeps them."""
    global _handle
    from gather_radix_top_gb300 import kvo
    if _handle is None:
        _handle = kvo.Context(layers=1, history_cap=64, hot_rows=64)
    st["cache"] = kvo.Cache(rows=st.get("rows"), keys=st.get("keys"), key_scales=st.get("key_scales"),
                            block_rows=st["block_rows"], table=st["table"])
    return st["cache"]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        cache = state.get("cache") or _open(state)
        if op == "append":
            kv = state["kv"]
            _handle.append_tokens(cache, kv[:, :LATENT], kv[:, LATENT:], state["pos"], state["inv_freq"],
                                  seq=state["seq"], key=state.get("key"), interleaved=case["interleaved"],
                                  out_bf16=state["values"])
            return _appended(state, state["values"])
        if op == "score":
            return _handle.index_scores(cache, state["q"], state["w"], state["lens"], case["length"],
                                        block=case["block"], out=state["out"])
        return _handle.attend(cache, state["q"], state["lens"], state["scale"], rows=case["length"],
                              sel=state["sel"], sel_block=case["sel_block"], out=state["out"], lse=state["lse"])
    return {"append": _append, "score": _score, "attend": _attend}[op](state)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, one sequence or token group at a time."""
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "score":
        return _exact_score(st)
    return _exact_attend(st)


def _row_numbers(st, s, n):
    """Cache row numbers of a sequence's positions 0 .. n - 1."""
    br = st["block_rows"]
    if st["table"] is None:
        return torch.arange(s * br, s * br + n, device="cuda")
    full = st["table"][s].long()[:, None] * br + torch.arange(br, device="cuda")[None, :]
    return full.reshape(-1)[:n]


def _exact_append(st):
    case, dev = st["case"], "cuda"
    n = case["tokens"]
    x = st["kv"].double()
    groups = x[:, :LATENT].reshape(n, GROUPS, 64)
    # every positive fp16, ascending: the first whose 127-fold reaches the group's largest value
    grid = torch.arange(0, 0x7C00, dtype=torch.int16, device=dev).view(torch.float16)
    at = torch.searchsorted(grid.double() * 127, groups.abs().amax(2).contiguous()).clamp(max=grid.numel() - 1)
    scale = grid.double()[at]
    q = torch.where(scale[..., None] > 0, torch.round(groups / scale[..., None].clamp(min=1e-30)),
                    torch.zeros((), dtype=torch.float64, device=dev)).clamp(-127, 127)
    theta = torch.outer(st["pos"].double(), st["inv_freq"].to(dev))
    z = torch.polar(torch.ones_like(theta), theta)
    part = x[:, LATENT:]
    pair = (part.reshape(n, ROPE // 2, 2) if case["interleaved"] else part.reshape(n, 2, ROPE // 2).transpose(1, 2))
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    turned = turned.reshape(n, ROPE) if case["interleaved"] else turned.transpose(1, 2).reshape(n, ROPE)
    total, br = st["rows"].shape[0], st["block_rows"]
    row = st["table"].long()[st["seq"].long(), torch.div(st["pos"].long(), br, rounding_mode="floor")] * br
    row = row + torch.remainder(st["pos"].long(), br)

    def put(v, width):
        full = torch.zeros(total, width, dtype=torch.float64, device=dev)
        full[row] = v
        return full

    out = [torch.cat([(q * scale[..., None]).reshape(n, LATENT), turned], 1), None, put(scale, GROUPS),
           put(turned, ROPE)]
    if case["key"] == "bf16":
        out.append(put(st["key"].double(), KEY))
    elif case["key"] == "e4m3":
        k = st["key"].double()
        m, e = torch.frexp(k.abs().amax(1))               # amax = m * 2^e, m in [0.5, 1): 448 = 0.875 * 2^9
        step = torch.exp2((e - 9 + (m > 0.875)).double()).clamp(min=2.0 ** -100)
        step = torch.where(m > 0, step, torch.full_like(step, 2.0 ** -100))
        out += [put(k / step[:, None], KEY), put(step[:, None], 1)[:, 0]]
    return out


def _exact_score(st):
    case, dev = st["case"], "cuda"
    n, q_n, block = case["length"], case["per_seq"], case["block"]
    out = torch.full((case["seqs"] * q_n, -(-n // block) * block), -math.inf, dtype=torch.float64, device=dev)
    for s in range(case["seqs"]):
        rows = _row_numbers(st, s, n)
        if case["dtype"] == "e4m3":
            keys = st["keys"].view(torch.uint8)[rows].view(DTYPES["e4m3"]).float().double()
            keys = keys * st["key_scales"][rows].double()[:, None]
        else:
            keys = st["keys"][rows].double()
        for t in range(s * q_n, (s + 1) * q_n):
            seen = int(st["lens"][t])
            dots = keys[:seen] @ st["q"][t].float().double().T
            out[t, :seen] = dots.clamp(min=0) @ st["w"][t].double()
    return out if block == 1 else out.reshape(out.shape[0], -1, block).amax(2)


def _exact_attend(st):
    case, dev = st["case"], "cuda"
    n, q_n, heads = case["length"], case["per_seq"], case["heads"]
    nq = case["seqs"] * q_n
    if nq * heads * (case["picked"] * case["sel_block"] or n) > 2 ** 28:
        return None
    out = torch.zeros(nq, heads, LATENT, dtype=torch.float64, device=dev)
    lse = torch.full((nq, heads), -math.inf, dtype=torch.float64, device=dev)
    for t in range(nq):
        rows, seen = _row_numbers(st, t // q_n, n), int(st["lens"][t])
        if st["sel"] is None:
            pick = torch.arange(seen, device=dev)
        else:
            b = case["sel_block"]
            pick = torch.cat([st["sel"][t].long() * b + i for i in range(b)])
            pick = pick[(pick >= 0) & (pick < seen)]
        if not pick.numel():
            continue
        raw = st["rows"][rows[pick]]
        q8 = raw[:, :LATENT].contiguous().view(torch.int8).double().reshape(-1, GROUPS, 64)
        sc = raw[:, LATENT:LATENT + 2 * GROUPS].contiguous().view(torch.float16).double()
        # a row stands for its dequantised bf16 values (int8 * fp16 is exact in 64 bits, rounded once)
        lat = (q8 * sc[..., None]).reshape(-1, LATENT).float().bfloat16().double()
        rp = raw[:, LATENT + 2 * GROUPS:].contiguous().view(torch.bfloat16).double()
        z = st["q"][t].double() @ torch.cat([lat, rp], 1).T * st["scale"]
        lse[t] = torch.logsumexp(z, 1)
        out[t] = torch.softmax(z, 1) @ lat
    return out, lse
