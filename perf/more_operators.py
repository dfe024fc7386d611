"""Prompt chunks over a paged cache, and caches shrunk by what attention looked at: how they are timed.

Three operators on one cache of 656-byte Q8G64 rows, held in blocks that a table maps (or one contiguous run per
sequence):

``chunk``    causal softmax attention of absorbed MLA queries for a ragged batch of new tokens, whose rows are the
             last ones of their sequences: token i of n sees the first length - n + 1 + i positions.
``weights``  the attention weight that a chunk's last tokens, all heads together, give to every cached position,
             from the log-sum-exps that the attention returned, added to what earlier chunks gave.
``shrink``   eviction: of every sequence the first, the last and the most attended positions, up to a budget, move
             into other blocks, in their order, with keys and weights.

``run`` computes them in elementary torch operations, or with the library's calls where ``own`` is set.
"""
import math

import torch

own = False

ROW, LATENT, ROPE, GROUPS, KEY = 656, 512, 64, 8, 128
E4M3 = torch.float8_e4m3fn
SCALE = 192 ** -0.5
LOGITS = 2 ** 28                     # of the plain form at a time

_handle = None


def listed():
    return [
        # the next token of one short stream, with few heads: the smallest call there is
        dict(name="chunk_one_token", op="chunk", seqs=1, tokens=1, heads=16, length=61, ragged=False, block_rows=0),
        # a verification round: four draft tokens of each of sixteen streams, over all that they hold
        dict(name="chunk_drafts", op="chunk", seqs=16, tokens=64, heads=16, length=8_192, ragged=False, block_rows=16),
        # a prompt of 4,096 tokens in one piece, into an empty cache
        dict(name="chunk_prompt_4k", op="chunk", seqs=1, tokens=4_096, heads=16, length=4_096, ragged=False,
             block_rows=16),
        # the last 512 tokens of a 50K prompt
        dict(name="chunk_512_of_50k", op="chunk", seqs=1, tokens=512, heads=64, length=50_023, ragged=False,
             block_rows=16),
        # pieces of several prompts in one call: uneven, one without tokens, one without rows, an odd head count
        dict(name="chunk_ragged", op="chunk", seqs=9, tokens=1_237, heads=20, length=12_345, ragged=True,
             block_rows=48),
        # a large piece with all heads of a large model
        dict(name="chunk_2048_of_16k", op="chunk", seqs=1, tokens=2_048, heads=128, length=16_384, ragged=False,
             block_rows=64),
        # one decode step of a served batch: every stream's token adds its weights
        dict(name="weights_decode", op="weights", seqs=64, tokens=64, window=0, heads=64, length=16_384, ragged=False,
             block_rows=16),
        # the last 32 tokens of a prompt's last chunk look back over 50K positions
        dict(name="weights_window_50k", op="weights", seqs=1, tokens=512, window=32, heads=64, length=50_023,
             ragged=False, block_rows=16),
        # all tokens of several uneven pieces
        dict(name="weights_ragged", op="weights", seqs=7, tokens=301, window=0, heads=20, length=20_011, ragged=True,
             block_rows=48),
        # a 50K session cut to 8,192 rows, with the keys of its indexer
        dict(name="shrink_50k", op="shrink", seqs=1, length=50_023, budget=8_192, first=4, last=64, ragged=False,
             key="e4m3", block_rows=16),
        # half of a million positions
        dict(name="shrink_1m", op="shrink", seqs=1, length=1_048_576, budget=524_288, first=4, last=512, ragged=False,
             key="e4m3", block_rows=16),
        # a batch of uneven sessions, some already within the budget
        dict(name="shrink_ragged", op="shrink", seqs=33, length=20_011, budget=1_021, first=1, last=61, ragged=True,
             key="bf16", block_rows=48),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "weights", "shrink"])
    if op == "shrink":
        seqs = _spread(rng, 1, 64)
        length = _spread(rng, 1, 1_048_576 // seqs)
        budget = _spread(rng, 1, max(1, length * 3 // 4))
        first = rng.choice([0, 1, 4]) if budget > 8 else 0
        return dict(op=op, seqs=seqs, length=length, budget=budget, first=first,
                    last=rng.randint(0, min(512, (budget - first) // 2)), ragged=rng.random() < 0.5,
                    key=rng.choice(["none", "bf16", "e4m3"]), block_rows=rng.choice([0, 16, 48, 64]))
    heads, ragged = rng.choice([1, 8, 16, 20, 64, 128]), rng.random() < 0.5
    seqs = _spread(rng, 1, 64)
    tokens = seqs * rng.choice([1, 1, 2, 4]) if rng.random() < 0.4 else _spread(rng, seqs, max(seqs, 4_096))
    # no more work than the largest listed case, and no more than 3 million rows
    most = min(262_144, 2 ** 31 // (tokens * heads), 3_000_000 // seqs)
    length = _spread(rng, 1, max(1, most))
    case = dict(op=op, seqs=seqs, tokens=tokens, heads=heads, length=length, ragged=ragged,
                block_rows=rng.choice([0, 16, 48, 64]))
    if op == "weights":
        case["window"] = rng.choice([0, 1, 16, 32, 64])
    return case


# ------------------------------------------------------------------ sizes
def _lengths(case):
    """The positions that each sequence holds, the new tokens' own among them."""
    n, s_n = case["length"], case["seqs"]
    if not case["ragged"]:
        return [n] * s_n
    return [0 if s_n > 2 and s == s_n - 1 else max(0, n - (n * ((s * 37) % 64)) // 96 - s % 5) for s in range(s_n)]


def _starts(case):
    """First token of each sequence, and the end of the last one's."""
    n, s_n = case["tokens"], case["seqs"]
    if not case["ragged"] or s_n == 1:
        return [n * s // s_n for s in range(s_n + 1)]
    share = [0 if s == 1 and s_n > 3 else 1 + (s * 5) % 7 for s in range(s_n)]
    return [n * sum(share[:s]) // sum(share) for s in range(s_n + 1)]


def _seen(case, window=0):
    """(sequence, token, visible positions) of every token that takes part."""
    starts, out = _starts(case), []
    for s, have in enumerate(_lengths(case)):
        n = starts[s + 1] - starts[s]
        for i in range(max(0, n - window) if window else 0, n):
            out.append((s, starts[s] + i, max(0, have - n + 1 + i)))
    return out


def work(case):
    lens, s_n = _lengths(case), case["seqs"]
    if case["op"] == "shrink":
        key = {"none": 0, "bf16": 2 * KEY, "e4m3": KEY + 4}[case["key"]]
        kept = sum(min(n, case["budget"]) for n in lens)
        # all weights, the kept rows and keys in and out, their positions and weights; a comparison a weight
        return dict(bytes=4 * sum(lens) + kept * (2 * (ROW + key) + 8) + 8 * s_n, flops=sum(lens))
    seen = _seen(case, case.get("window", 0))
    most = {}
    for s, _, n in seen:
        most[s] = max(most.get(s, 0), n)
    rows, pairs, heads = sum(most.values()), sum(n for _, _, n in seen), case["heads"]
    if case["op"] == "weights":
        return dict(bytes=rows * ROW + len(seen) * heads * (2 * (LATENT + ROPE) + 4) + 4 * sum(lens)
                    + 4 * s_n * case["length"], flops=pairs * heads * (2 * (LATENT + ROPE) + 3))
    return dict(bytes=rows * ROW + len(seen) * heads * (2 * (LATENT + ROPE) + 2 * LATENT + 4),
                flops=pairs * heads * (2 * (LATENT + ROPE) + 2 * LATENT + 4))


# ----------------------------------------------------------------- inputs
def _table(seqs, blocks, g):
    """A shuffled block table and the number of blocks behind it."""
    total = seqs * blocks + 3
    ids = torch.randperm(total, generator=g, device="cuda")[:seqs * blocks]
    return ids.view(seqs, blocks).to(torch.int32), total


def _rows(n, g):
    rows = torch.empty(n, ROW, dtype=torch.uint8, device="cuda")
    rows.view(torch.int8)[:, :LATENT] = torch.randint(-127, 128, (n, LATENT), generator=g, device="cuda",
                                                      dtype=torch.int8)
    rows.view(torch.float16)[:, LATENT // 2:LATENT // 2 + GROUPS] = (
        torch.rand(n, GROUPS, generator=g, device="cuda") * 9e-3 + 1e-3).half()
    rows.view(torch.bfloat16)[:, LATENT // 2 + GROUPS:] = torch.randn(n, ROPE, generator=g, device="cuda").bfloat16()
    return rows


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s_n, n, dev = case["seqs"], case["length"], "cuda"
    br = case["block_rows"] or n
    state = dict(case=case, block_rows=br, lens=torch.tensor(_lengths(case), dtype=torch.int32, device=dev))
    state["table"], total = _table(s_n, -(-n // br), g) if case["block_rows"] else (None, s_n)
    state["rows"] = _rows(total * br, g)

    if case["op"] == "shrink":
        # what some hundred tokens left behind: a few positions with most of it, many with next to nothing, some
        # with exactly nothing
        w = torch.exp(3 * torch.randn(s_n, n, generator=g, device=dev) - 4)
        state["weights"] = w * (torch.rand(s_n, n, generator=g, device=dev) > 0.1)
        budget = case["budget"]
        to_br = case["block_rows"] or budget
        state["to_table"], to_total = _table(s_n, -(-budget // to_br), g) if case["block_rows"] else (None, s_n)
        state["to_block_rows"] = to_br
        state["to_rows"] = torch.zeros(to_total * to_br, ROW, dtype=torch.uint8, device=dev)
        if case["key"] != "none":
            keys = torch.randn(total * br, KEY, generator=g, device=dev)
            state["keys"] = keys.to(E4M3) if case["key"] == "e4m3" else keys.bfloat16()
            if case["key"] == "e4m3":
                state["key_scales"] = torch.exp2(torch.randint(-6, 1, (total * br,), generator=g, device=dev).float())
                state["to_keys"] = torch.zeros(to_total * to_br, KEY, dtype=torch.uint8, device=dev).view(E4M3)
                state["to_key_scales"] = torch.zeros(to_total * to_br, device=dev)
            else:
                state["to_keys"] = torch.zeros(to_total * to_br, KEY, dtype=torch.bfloat16, device=dev)
        state["kept"] = torch.empty(s_n, budget, dtype=torch.int32, device=dev)
        state["new_lens"] = torch.empty(s_n, dtype=torch.int32, device=dev)
        state["to_weights"] = torch.empty(s_n, budget, device=dev)
        return state

    tokens, heads = case["tokens"], case["heads"]
    state["starts"] = torch.tensor(_starts(case), dtype=torch.int32, device=dev)
    # some heads look at few positions, some at nearly all
    gain = torch.exp(0.7 * torch.randn(1, heads, 1, generator=g, device=dev) + 0.5)
    state["q"] = (torch.randn(tokens, heads, LATENT + ROPE, generator=g, device=dev) * gain).bfloat16()
    if case["op"] == "chunk":
        state["out"] = torch.empty(tokens, heads, LATENT, dtype=torch.bfloat16, device=dev)
        state["lse"] = torch.empty(tokens, heads, device=dev)
        return state
    # the log-sum-exps as the attention has returned them, and what earlier chunks gave
    state["lse"] = torch.full((tokens, heads), -math.inf, device=dev)
    for at, z, _, _ in _logits(state, case["window"]):
        state["lse"][at] = torch.logsumexp(z, 2)
    state["carry"] = torch.exp(2 * torch.randn(s_n, n, generator=g, device=dev) - 3)
    state["keep"] = 0.96875
    state["out"] = torch.empty(s_n, n, device=dev)
    return state


# -------------------------------------------------------------- plain form
def _places(table, block_rows, seq, pos):
    """The cache rows of a sequence's positions."""
    if table is None:
        return seq * block_rows + pos
    return table[seq].long()[pos // block_rows] * block_rows + pos % block_rows


def _values_of_rows(rows):
    """What rows stand for, as the cache's dequantised rows have it: bf16 of int8 * scale, and the position part."""
    q = rows[..., :LATENT].contiguous().view(torch.int8).float()
    scale = rows[..., LATENT:LATENT + 2 * GROUPS].contiguous().view(torch.float16).float()
    latent = (q.unflatten(-1, (GROUPS, 64)) * scale[..., None]).flatten(-2).bfloat16()
    return latent.float(), rows[..., LATENT + 2 * GROUPS:].contiguous().view(torch.bfloat16).float()


def _logits(st, window=0):
    """(tokens, masked logits [tokens, heads, positions], latents, sequence) of one group of tokens after the other."""
    case, starts = st["case"], _starts(st["case"])
    for s, have in enumerate(_lengths(case)):
        n = starts[s + 1] - starts[s]
        take = min(n, window) if window else n
        if have == 0 or take == 0:
            continue
        pos = torch.arange(have, device="cuda")
        latent, rope = _values_of_rows(st["rows"][_places(st["table"], st["block_rows"], s, pos)])
        step = max(1, LOGITS // (have * case["heads"]))
        for i in range(n - take, n, step):
            j = min(n, i + step)
            at = slice(starts[s] + i, starts[s] + j)
            q = st["q"][at].float()
            z = (q[..., :LATENT] @ latent.T + q[..., LATENT:] @ rope.T) * SCALE
            last = have - n + torch.arange(i, j, device="cuda")
            yield at, z.masked_fill_(pos > last[:, None, None], -math.inf), latent, s


def _chunk(st):
    out, lse = torch.zeros_like(st["out"]), torch.full_like(st["lse"], -math.inf)
    for at, z, latent, _ in _logits(st):
        top = z.amax(2, keepdim=True)
        top = torch.where(top.isfinite(), top, 0.0)
        p = torch.exp(z - top)
        total = p.sum(2, keepdim=True)
        out[at] = ((p @ latent) / torch.where(total > 0, total, 1.0)).bfloat16()
        lse[at] = torch.log(total[..., 0]) + top[..., 0]
    return out, lse


def _weights(st):
    lens = st["lens"].long()
    out = st["keep"] * st["carry"]
    for at, z, _, s in _logits(st, st["case"]["window"]):
        lse = st["lse"][at][..., None]
        p = torch.where(lse == -math.inf, 0.0, torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)))
        out[s, :z.shape[2]] += p.sum((0, 1))
    return out.masked_fill_(torch.arange(out.shape[1], device="cuda") >= lens[:, None], 0.0)


def _shrink(st):
    case = st["case"]
    kept, new_lens, to_weights = st["kept"], st["new_lens"], st["to_weights"]
    kept.fill_(-1)
    to_weights.zero_()
    for s, have in enumerate(_lengths(case)):
        n = min(have, case["budget"])
        order = st["weights"][s, :have].clone()
        order[:case["first"]] = math.inf
        order[max(0, have - case["last"]):] = math.inf
        pick = order.sort(descending=True, stable=True).indices[:n].sort().values
        new_lens[s] = n
        kept[s, :n] = pick
        to_weights[s, :n] = st["weights"][s, pick]
        src = _places(st["table"], st["block_rows"], s, pick)
        dst = _places(st["to_table"], st["to_block_rows"], s, torch.arange(n, device="cuda"))
        for name in ("rows", "keys", "key_scales"):
            if name in st:
                bits = torch.uint8 if st[name].dtype == E4M3 else st[name].dtype
                st["to_" + name].view(bits)[dst] = st[name].view(bits)[src]
    return _shrunk(st)


def _shrunk(st):
    rows = st["to_rows"]
    out = [st["kept"], st["new_lens"], st["to_weights"], rows.view(torch.int8)[:, :LATENT],
           rows.view(torch.float16)[:, LATENT // 2:LATENT // 2 + GROUPS],
           rows.view(torch.bfloat16)[:, LATENT // 2 + GROUPS:]]
    return out + [st[k] for k in ("to_keys", "to_key_scales") if k in st]


# ---------------------------------------------------------- the library's calls
def _open(st):
    """The context (one for all) and the views of this state's caches, kept as a program keeps them."""
    global _handle
    from gather_radix_top_gb300 import kvo
    if _handle is None:
        _handle = kvo.Context(layers=1, history_cap=64, hot_rows=64)
    st["cache"] = kvo.Cache(rows=st["rows"], keys=st.get("keys"), key_scales=st.get("key_scales"),
                            block_rows=st["block_rows"], table=st["table"])
    if "to_rows" in st:
        st["to"] = kvo.Cache(rows=st["to_rows"], keys=st.get("to_keys"), key_scales=st.get("to_key_scales"),
                             block_rows=st["to_block_rows"], table=st["to_table"])
    return st["cache"]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        cache = state.get("cache") or _open(state)
        if op == "chunk":
            return _handle.attend_chunk(cache, state["q"], state["starts"], state["lens"], SCALE, case["length"],
                                        out=state["out"], lse=state["lse"])
        if op == "weights":
            return _handle.attention_weights(cache, state["q"], state["starts"], state["lens"], state["lse"], SCALE,
                                             case["length"], window=case["window"], carry=state["carry"],
                                             keep=state["keep"], out=state["out"])
        _handle.shrink_cache(cache, state["to"], state["weights"], state["lens"], case["budget"], first=case["first"],
                             last=case["last"], kept=state["kept"], new_lens=state["new_lens"],
                             to_weights=state["to_weights"])
        return _shrunk(state)
    return {"chunk": _chunk, "weights": _weights, "shrink": _shrink}[op](state)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, token by token or row by row."""
    st = prepare(case, seed)
    if case["op"] == "shrink":
        return _exact_shrink(st)
    window = case.get("window", 0)
    seen = _seen(case, window)
    if case["heads"] * sum(n for _, _, n in seen) > 2 ** 31 or len(seen) > 8_192:
        return None
    dev = "cuda"
    out = torch.zeros(case["tokens"], case["heads"], LATENT, dtype=torch.float64, device=dev)
    lse = torch.full((case["tokens"], case["heads"]), -math.inf, dtype=torch.float64, device=dev)
    mass = torch.zeros(case["seqs"], case["length"], dtype=torch.float64, device=dev)
    if window or case["op"] == "weights":
        for s, have in enumerate(_lengths(case)):
            mass[s, :have] = st["keep"] * st["carry"][s, :have].double()
    held = (None, None, None)
    for s, t, n in seen:
        if n == 0:
            continue
        if held[0] != s:
            raw = st["rows"][_numbers(st["table"], st["block_rows"], s, _lengths(case)[s])]
            q8 = raw[:, :LATENT].contiguous().view(torch.int8).double().reshape(-1, GROUPS, 64)
            sc = raw[:, LATENT:LATENT + 2 * GROUPS].contiguous().view(torch.float16).double()
            # a row stands for its dequantised bf16 values (int8 * fp16 is exact in 64 bits, rounded once)
            lat = (q8 * sc[..., None]).reshape(-1, LATENT).float().bfloat16().double()
            rope = raw[:, LATENT + 2 * GROUPS:].contiguous().view(torch.bfloat16).double()
            held = (s, lat, torch.cat([lat, rope], 1))
        z = st["q"][t].double() @ held[2][:n].T * SCALE
        if case["op"] == "weights":
            mass[s, :n] += torch.exp(z - st["lse"][t].double()[:, None]).sum(0)
            continue
        lse[t] = torch.logsumexp(z, 1)
        out[t] = torch.softmax(z, 1) @ held[1][:n]
    return mass if case["op"] == "weights" else (out, lse)


def _numbers(table, br, s, n):
    """Cache row numbers of a sequence's positions 0 .. n - 1."""
    if table is None:
        return torch.arange(s * br, s * br + n, device="cuda")
    return (table[s].long()[:, None] * br + torch.arange(br, device="cuda")[None, :]).reshape(-1)[:n]


def _exact_shrink(st):
    case, dev = st["case"], "cuda"
    budget, s_n = case["budget"], case["seqs"]
    kept = torch.full((s_n, budget), -1, dtype=torch.int64, device=dev)
    lens = torch.zeros(s_n, dtype=torch.int64, device=dev)
    weights = torch.zeros(s_n, budget, dtype=torch.float64, device=dev)
    src, dst = [], []
    for s, have in enumerate(_lengths(case)):
        pos = torch.arange(have, device=dev)
        fixed = (pos < case["first"]) | (pos >= have - case["last"])
        w = st["weights"][s, :have].double()
        if have > budget:
            # everything above the smallest weight that still gets in, and as many at it, from the front, as fit
            free = budget - int(fixed.sum())
            border = w[~fixed].kthvalue(int((~fixed).sum()) - free + 1).values if free else math.inf
            above = ~fixed & (w > border)
            level = ~fixed & (w == border)
            level &= level.cumsum(0) <= free - above.sum()
            pos = pos[fixed | above | level]
        n = lens[s] = len(pos)
        kept[s, :n] = pos
        weights[s, :n] = w[pos]
        src.append(_numbers(st["table"], st["block_rows"], s, have)[pos])
        dst.append(_numbers(st["to_table"], st["to_block_rows"], s, int(n)))
    src, dst = torch.cat(src), torch.cat(dst)
    total = st["to_rows"].shape[0]

    def move(x, width):
        full = torch.zeros(total, width, dtype=torch.float64, device=dev)
        full[dst] = x.reshape(-1, width)[src].double()
        return full

    rows = st["rows"]
    out = [kept, lens, weights, move(rows[:, :LATENT].view(torch.int8), LATENT),
           move(rows[:, LATENT:LATENT + 2 * GROUPS].contiguous().view(torch.float16), GROUPS),
           move(rows[:, LATENT + 2 * GROUPS:].contiguous().view(torch.bfloat16), ROPE)]
    if "keys" in st:
        out.append(move(st["keys"].float(), KEY))
    if "key_scales" in st:
        out.append(move(st["key_scales"], 1)[:, 0])
    return out
