"""kvo_append_tokens, kvo_index_scores and kvo_attend against the 64-bit oracle.

Tolerances, from the number formats alone (u = 2^-24, half a step of fp32;
2^-8, half a step of bf16):
  rotated values   2^-8 |x| for the one rounding, and 8 u (|a| + |b|) for the
                   reduced angle, the sine and cosine and the three products;
  scores           every product of the keys' types is exact in fp32; a sum of
                   128 + 64 terms, each step off by at most 2 u of the sum of
                   magnitudes (an accumulator may truncate), the factors
                   2 steps more;
  lse              the logits' error (576 steps of 2 u of the magnitudes), the
                   exponentials and the logarithm 16 u, a blocked sum 2 u for
                   each of n / 128 + 32 steps, and 2 u of its size;
  out              2^-8 |out| for its rounding, and for the sum of p |v| the
                   weights' rounding 2^-8, twice the logits' error and the
                   steps of the sum as above.
Quantised values, their scales and factors have to be equal.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kvo_sparse_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INV_FREQ = 10_000.0 ** (-np.arange(0, 64, 2) / 64)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ctx():
    from gather_radix_top_gb300 import build, kvo
    build.build()
    c = kvo.Context(1, 64, 64)
    yield c
    c.close()


@pytest.fixture(scope="module")
def kvo():
    from gather_radix_top_gb300 import kvo as K
    return K


def dev(x, dtype=None):
    t = torch.as_tensor(x)
    return (t if dtype is None else t.to(dtype)).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def block_table(rng, sequences, blocks, spare=2):
    total = sequences * blocks + spare
    return rng.permutation(total)[:sequences * blocks].reshape(sequences, blocks).astype(np.int32), total


def random_rows(rng, n, scale=(1e-3, 1e-2)):
    rows = rng.integers(0, 256, (n, 656), dtype=np.uint8)
    rows[:, :512][rows[:, :512] == 128] = 0
    rows[:, 512:528] = rng.uniform(*scale, (n, 8)).astype(np.float16).view(np.uint8)
    rows[:, 528:] = np.ascontiguousarray(O.bf16_bits(rng.standard_normal((n, 64)))).view(np.uint8)
    return rows


# -------------------------------------------------------------------- append
def append_case(kvo, ctx, rng, dtype, n, interleaved, key, block_rows, seqs=None, pos=None, sequences=None, spread=3.0,
                x=None, ld=None):
    sequences = sequences or max(1, n)
    seqs = np.arange(n, dtype=np.int32) if seqs is None else np.asarray(seqs, np.int32)
    pos = rng.integers(0, 3 * block_rows, n).astype(np.int32) if pos is None else np.asarray(pos, np.int32)
    table, blocks = block_table(rng, sequences, 3)
    wide = ld or 576
    kv = rng.standard_normal((max(n, 1), wide)) * np.exp(rng.normal(0, spread, (max(n, 1), wide)))
    if x is not None:
        kv[:x.shape[0], :x.shape[1]] = x
    kv = dev(kv, TYPES[dtype])[:n]
    kk = dev(rng.standard_normal((n, 128)) * np.exp(rng.normal(0, spread, (n, 128))), TYPES[dtype])
    R = blocks * block_rows
    rows = torch.full((R, 656), 0x5A, dtype=torch.uint8, device="cuda")
    keys = scales = None
    if key == "bf16":
        keys = torch.full((R, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    elif key == "e4m3":
        keys = torch.full((R, 128), 0x22, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.full((R,), 5.0, device="cuda")
    cache = kvo.Cache(rows=rows, keys=keys, key_scales=scales, block_rows=block_rows, table=dev(table))
    values = torch.full((n, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    ctx.append_tokens(cache, kv[:, :512], kv[:, 512:576], dev(pos), INV_FREQ, seq=dev(seqs),
                      key=kk if key != "none" else None, interleaved=interleaved, out_bf16=values)
    status = ctx.sync()
    return dict(kv=f64(kv), kk=f64(kk), rows=rows.cpu().numpy(), keys=keys, scales=scales, table=table, blocks=blocks,
                seqs=seqs, pos=pos, values=values, status=status, sequences=sequences)


def check_append(kvo, r, dtype, interleaved, key, block_rows):
    want_rows = np.full_like(r["rows"], 0x5A)
    touched, bad = set(), False
    got_values = f64(r["values"])
    for i, (s, p) in enumerate(zip(r["seqs"], r["pos"])):
        if s < 0:
            assert (got_values[i] == 7.0).all()
            continue
        at = None
        if s < r["sequences"] and p >= 0:
            at = O.row_of(r["table"], r["blocks"], block_rows, r["sequences"], int(s), int(p))
        if at is None:
            bad = True
            assert not got_values[i].any()
            continue
        touched.add(at)
        row = r["rows"][at]
        for g in range(8):
            q, bits = O.latent_group(r["kv"][i, 64 * g:64 * g + 64])
            assert int(row[512 + 2 * g:514 + 2 * g].view(np.uint16)[0]) == bits
            assert np.array_equal(row[64 * g:64 * g + 64].view(np.int8), q), (i, g)
        latent, rope = O.row_values(row)
        assert np.array_equal(latent, got_values[i, :512], equal_nan=True)
        assert np.array_equal(rope, got_values[i, 512:], equal_nan=True)
        x = r["kv"][i, 512:576]
        exact = O.rotate(x, int(p), INV_FREQ, interleaved)
        pair = np.abs(x[0::2]) + np.abs(x[1::2]) if interleaved else np.abs(x[:32]) + np.abs(x[32:])
        pair = np.repeat(pair, 2) if interleaved else np.tile(pair, 2)
        assert (np.abs(rope - exact) <= 2.0 ** -8 * np.abs(exact) + 8 * U * pair + 2.0 ** -133).all(), i
        if key == "bf16":
            got = r["keys"][at].view(torch.int16).cpu().numpy().view(np.uint16)
            assert np.array_equal(got, O.bf16_bits(r["kk"][i]))
        elif key == "e4m3":
            want, factor = O.key_e4m3(r["kk"][i])
            assert float(r["scales"][at]) == factor
            assert np.array_equal(r["keys"][at].view(torch.uint8).cpu().numpy(), want)
        want_rows[at] = row
    assert np.array_equal(r["rows"], want_rows)              # nothing else was written
    rest = [i for i in range(len(r["rows"])) if i not in touched]
    if key == "e4m3":
        assert (r["keys"].view(torch.uint8)[rest] == 0x22).all() and (r["scales"][rest] == 5.0).all()
    elif key == "bf16":
        assert (r["keys"][rest] == 3.0).all()
    assert r["status"] == (kvo.KVO_ERANGE if bad else kvo.KVO_OK)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("key", ["none", "bf16", "e4m3"])
@pytest.mark.parametrize("n,block_rows,interleaved", [(1, 16, True), (7, 5, False), (33, 16, True), (65, 1, False)])
def test_append(kvo, ctx, dtype, key, n, block_rows, interleaved):
    rng = np.random.default_rng([n, block_rows, len(dtype), ord(key[0])])
    spread = 1.0 if dtype == "fp16" else 3.0
    r = append_case(kvo, ctx, rng, dtype, n, interleaved, key, block_rows, spread=spread, ld=640 if n == 7 else None)
    check_append(kvo, r, dtype, interleaved, key, block_rows)


def test_append_nothing(kvo, ctx):
    r = append_case(kvo, ctx, np.random.default_rng(1), "bf16", 0, True, "e4m3", 16)
    assert (r["rows"] == 0x5A).all() and r["status"] == kvo.KVO_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_edge_values(kvo, ctx, dtype):
    """Groups of zeros, of values that no scale holds, next to rounding borders, infinite and NaN."""
    rng = np.random.default_rng(9)
    x = rng.standard_normal((8, 512))
    x[0] = 0.0
    x[1, 64:128] = 0.0
    x[1, 70] = 2.0 ** -60
    x[2, 0] = 1e30
    x[3, 5], x[3, 200], x[3, 400] = np.inf, np.nan, -np.inf
    x[4] = np.tile(np.arange(64) - 32 + 0.5, 8) * 2.0 ** -7   # ties of a power-of-two scale
    x[4, ::64] = 127 * 2.0 ** -7
    s = float(np.float16(0.0037))
    x[5] = (np.arange(512) % 127 + 0.5) * s                   # as near to ties as the type gets
    x[5, ::64] = 127 * s
    x[6] = np.nextafter(np.float32((np.arange(512) % 127 + 0.5)) * np.float32(s), np.float32(0))
    x[6, ::64] = 127 * s
    x[7] *= 2.0 ** -22                                        # subnormal scales
    r = append_case(kvo, ctx, rng, dtype, 8, True, "e4m3", 16, x=x)
    check_append(kvo, r, dtype, True, "e4m3", 16)


def test_append_key_edges(kvo, ctx):
    rng = np.random.default_rng(10)
    kk = rng.standard_normal((6, 128)).astype(np.float32)
    kk[0] = 0.0
    kk[1] = 0.0
    kk[1, 3] = 448 * 2.0 ** -5                                # exactly the largest e4m3 at its factor
    kk[2] = 0.0
    kk[2, 3] = np.nextafter(np.float32(448 * 2.0 ** -5), np.float32(1e9))
    kk[3, 7] = np.inf
    kk[4, 0] = np.nan
    kk[5] = np.float32(2.0 ** -140)
    rows = torch.zeros(6, 656, dtype=torch.uint8, device="cuda")
    keys = torch.zeros(6, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros(6, device="cuda")
    cache = kvo.Cache(rows=rows, keys=keys, key_scales=scales, block_rows=1)
    kv = torch.randn(6, 576, device="cuda")
    ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], torch.zeros(6, dtype=torch.int32, device="cuda"), INV_FREQ,
                      key=dev(kk))
    assert ctx.sync() == kvo.KVO_OK
    for i in range(6):
        want, factor = O.key_e4m3(kk[i])
        assert np.array_equal(float(scales[i]), factor, equal_nan=True)
        assert np.array_equal(keys[i].view(torch.uint8).cpu().numpy(), want), i


@pytest.mark.parametrize("interleaved", [True, False])
def test_append_far_positions(kvo, ctx, interleaved):
    """Angles of positions up to 2^31 - 1 (a table whose last entry alone is used)."""
    rng = np.random.default_rng(11)
    pos = np.array([0, 1, 65_535, 1_048_575, 16_777_217, 2 ** 31 - 1], np.int32)
    rows = torch.zeros(6, 656, dtype=torch.uint8, device="cuda")
    kv = rng.standard_normal((6, 576)).astype(np.float32)
    for i, p in enumerate(pos):
        block = 2 ** 30
        table = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
        big = kvo.Cache(rows=rows[i:i + 1], block_rows=1, table=table)
        # one block of 2^30 rows a table entry, of which only the addressed row exists: shift the base
        big.c.block_rows, big.c.blocks = block, 1
        table[0, int(p) // block] = 0
        big.c.rows = rows.data_ptr() + i * 656 - (int(p) % block) * 656
        ctx.append_tokens(big, dev(kv[i:i + 1, :512]), dev(kv[i:i + 1, 512:]), dev(pos[i:i + 1]), INV_FREQ,
                          interleaved=interleaved)
    assert ctx.sync() == kvo.KVO_OK
    out = rows.cpu().numpy()
    for i, p in enumerate(pos):
        x = kv[i, 512:].astype(np.float64)
        exact = O.rotate(x, int(p), INV_FREQ, interleaved)
        pair = np.abs(x[0::2]) + np.abs(x[1::2]) if interleaved else np.abs(x[:32]) + np.abs(x[32:])
        pair = np.repeat(pair, 2) if interleaved else np.tile(pair, 2)
        rope = O.row_values(out[i])[1]
        assert (np.abs(rope - exact) <= 2.0 ** -8 * np.abs(exact) + 8 * U * pair).all(), p


def test_append_skips_padding_and_refuses_bad_places(kvo, ctx):
    rng = np.random.default_rng(12)
    r = append_case(kvo, ctx, rng, "bf16", 6, True, "e4m3", 4, seqs=[0, -1, 2, 3, 1, 0], pos=[0, 1, 11, 2, 7, 5],
                    sequences=4)
    check_append(kvo, r, "bf16", True, "e4m3", 4)
    assert r["status"] == kvo.KVO_OK
    r = append_case(kvo, ctx, rng, "bf16", 6, True, "e4m3", 4, seqs=[0, 4, 2, 3, 1, 0], pos=[0, 1, 12, -2, 7, 5],
                    sequences=4)
    check_append(kvo, r, "bf16", True, "e4m3", 4)
    assert r["status"] == kvo.KVO_ERANGE


def test_append_bad_table_entries(kvo, ctx):
    rows = torch.full((8, 656), 0x5A, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[-1, 2 ** 31 - 1], [2, 0]], dtype=torch.int32, device="cuda")
    cache = kvo.Cache(rows=rows, block_rows=4, table=table)
    kv = torch.randn(3, 576, device="cuda")
    seq = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([1, 5, 2], dtype=torch.int32, device="cuda")
    ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], pos, INV_FREQ, seq=seq)
    assert ctx.sync() == kvo.KVO_ERANGE
    assert (rows == 0x5A).all()


# --------------------------------------------------------------------- score
def score_inputs(rng, nq, heads, keys_n, dtype):
    q = dev(rng.standard_normal((nq, heads, 128)), torch.float32)
    k = dev(rng.standard_normal((keys_n, 128)), torch.float32)
    if dtype == "e4m3":
        q, k = q.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn)
        scales = torch.exp2(dev(rng.integers(-6, 2, keys_n), torch.float32))
    else:
        q, k, scales = q.bfloat16(), k.bfloat16(), None
    w = dev(rng.standard_normal((nq, heads)), torch.float32)
    return q, k, scales, w


def check_scores(got, q, k, scales, w, rows, lens, n, block):
    factors = np.ones(k.shape[0]) if scales is None else f64(scales)
    heads = q.shape[1]
    padded = [list(r) + [None] * (n - len(r)) for r in rows]
    want, size = O.index_scores(f64(q), f64(w), f64(k), factors, padded, lens, block)
    got = f64(got)
    assert got.shape == want.shape
    fin = np.isfinite(want)
    assert np.array_equal(np.isneginf(got), np.isneginf(want)) and np.array_equal(np.isnan(got), np.isnan(want))
    tol = (128 + heads + 2) * 2 * U * size
    assert (np.abs(got - want)[fin] <= tol[fin]).all(), float((np.abs(got - want)[fin] - tol[fin]).max())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("sequences,per_seq,heads,n,block,block_rows", [
    (1, 1, 1, 1, 1, 1), (1, 1, 64, 130, 1, 16), (2, 4, 64, 257, 1, 16), (3, 2, 24, 300, 16, 48), (1, 1, 128, 129, 64, 7),
    (2, 3, 100, 200, 128, 16), (1, 7, 40, 140, 32, 64), (1, 1, 8, 1000, 2, 16), (5, 1, 17, 128, 4, 128)])
def test_scores(kvo, ctx, dtype, sequences, per_seq, heads, n, block, block_rows):
    rng = np.random.default_rng([sequences, per_seq, heads, n, len(dtype)])
    nq, blocks = sequences * per_seq, -(-n // block_rows)
    table, total = block_table(rng, sequences, blocks)
    q, k, scales, w = score_inputs(rng, nq, heads, total * block_rows, dtype)
    lens = rng.integers(0, n + 1, nq)
    lens[0] = n
    if nq > 2:
        lens[1] = 0
    if nq > 3:
        lens[2] = -3
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=block_rows, table=dev(table))
    got = ctx.index_scores(cache, q, w, dev(lens, torch.int32), n, block=block)
    assert ctx.sync() == kvo.KVO_OK
    rows = [[O.row_of(table, total, block_rows, sequences, t // per_seq, p) for p in range(n)] for t in range(nq)]
    check_scores(got, q, k, scales, w, rows, lens, n, block)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lengths", ["uneven", "one long", "none"])
@pytest.mark.parametrize("sequences,per_seq,heads,n,block,block_rows", [
    (90, 1, 16, 700, 1, 16), (40, 5, 64, 300, 1, 16), (100, 1, 64, 1000, 16, 16), (65, 4, 24, 500, 64, 48),
    (1100, 1, 8, 150, 1, 16), (160, 1, 128, 129, 128, 7), (310, 1, 5, 2100, 2, 48), (600, 3, 100, 40, 1, 5)])
def test_scores_many_sequences(kvo, ctx, dtype, lengths, sequences, per_seq, heads, n, block, block_rows):
    """More tasks than half the SMs: CTAs go from one sequence to the next, past empty ones; blocks are shared."""
    rng = np.random.default_rng([sequences, per_seq, heads, n, len(dtype), len(lengths)])
    nq, blocks, total = sequences * per_seq, -(-n // block_rows), 60
    table = rng.integers(0, total, (sequences, blocks)).astype(np.int32)
    q, k, scales, w = score_inputs(rng, nq, heads, total * block_rows, dtype)
    if lengths == "uneven":
        lens = rng.integers(0, n + 1, nq)
        lens[rng.random(nq) < 0.2] = 0
        lens[:2 * per_seq] = 0
        lens[-1] = n
    elif lengths == "one long":
        lens = rng.integers(-1, 2, nq)
        lens[nq // 3] = n
        lens[-per_seq:] = 0
    else:
        lens = np.zeros(nq, np.int64)
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=block_rows, table=dev(table))
    out = torch.full((nq, -(-n // block) + 3), 3.0, device="cuda")[:, :-(-n // block)]
    got = ctx.index_scores(cache, q, w, dev(lens, torch.int32), n, block=block, out=out)
    assert ctx.sync() == kvo.KVO_OK
    at = np.arange(n)
    whole = table[:, at // block_rows].astype(np.int64) * block_rows + at % block_rows
    some = np.unique(np.concatenate([rng.choice(nq, min(nq, 60), replace=False), [0, nq // 3, nq - 1]]))
    check_scores(got[some], q[some], k, scales, w[some], [list(whole[t // per_seq]) for t in some], lens[some], n, block)
    columns = np.arange(-(-n // block))[None] * block                # every query: what is seen and what is not
    assert np.array_equal(np.isneginf(f64(got)), columns >= np.maximum(lens, 0)[:, None])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_scores_strides_and_contiguous_cache(kvo, ctx, dtype):
    rng = np.random.default_rng(21)
    nq, heads, n = 3, 20, 150
    wide, k, scales, w = score_inputs(rng, nq, 2 * heads, nq * n, dtype)
    q = wide[:, ::2]
    weights = torch.zeros(nq, 99, device="cuda")[:, 5:5 + heads]
    weights.copy_(w[:, :heads])
    out = torch.full((nq, 200), 3.0, device="cuda")
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=n)
    lens = np.array([150, 1, 77])
    ctx.index_scores(cache, q, weights, dev(lens, torch.int32), n, out=out[:, :n])
    assert ctx.sync() == kvo.KVO_OK
    assert (out[:, n:] == 3.0).all()
    rows = [list(range(t * n, (t + 1) * n)) for t in range(nq)]
    check_scores(out[:, :n], q, k, scales, weights, rows, lens, n, 1)


def test_scores_bad_pages(kvo, ctx):
    """Bad entries mask what they would hold; beyond a query's length they are not read."""
    rng = np.random.default_rng(22)
    q, k, scales, w = score_inputs(rng, 2, 16, 64, "e4m3")
    table = np.array([[1, -1, 3, 0], [2, 0, 77, 9999]], np.int32)
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=16, table=dev(table))
    for lens, want in (([64, 64], kvo.KVO_ERANGE), ([16, 32], kvo.KVO_OK)):
        got = ctx.index_scores(cache, q, w, dev(lens, torch.int32), 64)
        assert ctx.sync() == want
        rows = [[O.row_of(table, 4, 16, 2, t, p) for p in range(64)] for t in range(2)]
        check_scores(got, q, k, scales, w, rows, lens, 64, 1)
    # a table shorter than n
    short = kvo.Cache(keys=k, key_scales=scales, block_rows=16, table=dev(table[:1, :1]))
    got = ctx.index_scores(short, q[:1], w[:1], dev([40], torch.int32), 64)
    assert ctx.sync() == kvo.KVO_ERANGE
    assert torch.isneginf(got[0, 16:]).all() and torch.isfinite(got[0, :16]).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_scores_nan_keys(kvo, ctx, dtype):
    """A NaN stays in its own column, ranks lowest in a block, and masked keys are never looked at."""
    rng = np.random.default_rng(23)
    n, heads = 140, 16
    q, k, scales, w = score_inputs(rng, 1, heads, 256, dtype)
    if dtype == "bf16":
        k[5], k[130], k[150:] = math.nan, math.inf, math.nan
        k[130] *= q[0, 0].sign()
    else:
        scales[5], scales[150:] = math.nan, math.nan
        k.view(torch.uint8)[150:] = 0x7F
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=256)
    rows = [list(range(n))]
    for block in (1, 16):
        got = ctx.index_scores(cache, q, w, dev([n - 1], torch.int32), n, block=block)
        assert ctx.sync() == kvo.KVO_OK
        clean = f64(k).copy()
        if dtype == "e4m3" or block == 1:
            assert torch.isnan(got[0, 5]) if block == 1 else torch.isfinite(got[0, 0])
        assert torch.isneginf(got[0, n - 1]) if block == 1 else True
        keep = np.array([c for c in range(got.shape[1]) if c not in ((130,) if block == 1 else (8,))])
        if dtype == "bf16":
            clean[130] = 0.0
        factors = np.ones(256) if scales is None else f64(scales)
        want, size = O.index_scores(f64(q), f64(w), clean, factors, rows, [n - 1], block)
        g = f64(got)[:, keep]
        want, size = want[:, keep], size[:, keep]
        fin = np.isfinite(want)
        assert np.array_equal(np.isnan(g), np.isnan(want))
        assert (np.abs(g - want)[fin] <= ((128 + heads + 2) * 2 * U * size)[fin]).all()


def test_scores_feed_the_selection(kvo, ctx):
    """Scores of a short context select every visible position first, lower positions on ties."""
    rng = np.random.default_rng(24)
    q, k, scales, w = score_inputs(rng, 2, 32, 2 * 500, "e4m3")
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=500)
    lens = dev([500, 40], torch.int32)
    scores = ctx.index_scores(cache, q, w.abs(), lens, 500)
    idx = ctx.select_topk_batch(scores, 64)
    assert ctx.sync() == kvo.KVO_OK
    assert idx[1].tolist() == list(range(64))
    want = np.sort(np.argsort(-f64(scores[0]), kind="stable")[:64])
    assert np.array_equal(idx[0].cpu().numpy(), want)


# -------------------------------------------------------------------- attend
def check_attend(out, lse, q, scale, lists, heads):
    out, lse = f64(out), lse.cpu().numpy().astype(np.float64)
    for t, rows in enumerate(lists):
        want, want_lse, spread, size = O.attend(f64(q[t]), scale, rows)
        if not rows:
            assert not out[t].any() and np.isneginf(lse[t]).all(), t
            continue
        steps = len(rows) / 128 + 32
        logit = 2 * U * 576 * size
        tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2 * logit + 16 * U + 2 * U * steps)[:, None]
        assert (np.abs(out[t] - want) <= tol).all(), (t, float((np.abs(out[t] - want) / tol).max()))
        tol = logit + 16 * U + 2 * U * steps + 2 * U * np.abs(want_lse)
        assert (np.abs(lse[t] - want_lse) <= tol).all(), (t, float((np.abs(lse[t] - want_lse) / tol).max()))


def attend_case(kvo, ctx, rng, sequences, per_seq, heads, n, sel_block, picked, block_rows, lens=None, scale=192 ** -0.5,
                sel=None, rows_scale=(1e-3, 1e-2)):
    nq = sequences * per_seq
    blocks = -(-n // block_rows) if n else 1
    table, total = block_table(rng, sequences, blocks)
    rows = random_rows(rng, total * block_rows, rows_scale)
    q = dev(rng.standard_normal((nq, heads, 576)), torch.bfloat16)
    if lens is None:
        lens = rng.integers(0, n + 1, nq)
        lens[0] = n
        if nq > 2:
            lens[1] = 0
    if sel is None and picked is not None:
        units = -(-n // sel_block)
        sel = np.stack([np.sort(rng.choice(units, picked, replace=False)) for _ in range(nq)]).astype(np.int32)
    cache = kvo.Cache(rows=dev(rows), block_rows=block_rows, table=dev(table))
    out, lse = ctx.attend(cache, q, dev(lens, torch.int32), scale, rows=n, sel=None if sel is None else dev(sel),
                          sel_block=sel_block)
    assert ctx.sync() == kvo.KVO_OK
    lists = []
    for t in range(nq):
        pos = O.positions_of(None if sel is None else sel[t], sel_block, int(lens[t]), n)
        lists.append([rows[O.row_of(table, total, block_rows, sequences, t // per_seq, p)] for p in pos])
    check_attend(out, lse, q, scale, lists, heads)


@pytest.mark.parametrize("sequences,per_seq,heads,n,block_rows", [
    (1, 1, 1, 1, 1), (1, 1, 64, 128, 16), (1, 1, 16, 127, 16), (1, 1, 128, 129, 48), (3, 2, 20, 300, 16),
    (2, 1, 100, 513, 64), (1, 4, 33, 260, 7), (1, 1, 64, 5000, 16), (40, 1, 8, 70, 16)])
def test_attend_whole_sequences(kvo, ctx, sequences, per_seq, heads, n, block_rows):
    rng = np.random.default_rng([sequences, per_seq, heads, n])
    attend_case(kvo, ctx, rng, sequences, per_seq, heads, n, 1, None, block_rows)


@pytest.mark.parametrize("sequences,per_seq,heads,n,sel_block,picked,block_rows", [
    (1, 1, 64, 4000, 1, 2048, 16), (2, 2, 20, 1000, 1, 129, 48), (1, 1, 7, 50, 1, 1, 16), (3, 1, 64, 700, 16, 23, 16),
    (1, 3, 128, 1000, 64, 9, 16), (2, 1, 32, 900, 128, 5, 7), (1, 1, 48, 333, 2, 100, 64)])
def test_attend_selected(kvo, ctx, sequences, per_seq, heads, n, sel_block, picked, block_rows):
    rng = np.random.default_rng([sequences, per_seq, heads, n, sel_block])
    attend_case(kvo, ctx, rng, sequences, per_seq, heads, n, sel_block, picked, block_rows)


@pytest.mark.parametrize("sequences,heads", [(18, 64), (20, 64), (24, 50), (28, 64), (18, 128), (45, 64), (70, 33), (40, 20),
                                             (60, 16)])
@pytest.mark.parametrize("listed", [False, True])
def test_attend_a_few_splits_a_query(kvo, ctx, sequences, heads, listed):
    """Between 18 and 76 queries share the SMs, so that two to eight CTAs join their parts of each; some parts are
    empty (whole sequences of a few rows) or see nothing (listed positions past the length)."""
    rng = np.random.default_rng([sequences, heads, listed])
    n = 640
    lens = rng.integers(0, n + 1, sequences)
    lens[:6] = n, 0, 1, 17, 81, 320
    attend_case(kvo, ctx, rng, sequences, 1, heads, n, 1, 600 if listed else None, 16, lens=lens)


@pytest.mark.parametrize("sequences,heads,n", [(10, 64, 1100), (6, 64, 2048), (4, 64, 3000), (1, 64, 9000), (1, 128, 6000),
                                               (3, 128, 1700)])
def test_attend_many_splits_a_query(kvo, ctx, sequences, heads, n):
    """About 15, 25, 38 and 76 to 140 splits; a query of one row leaves most of its splits empty."""
    rng = np.random.default_rng([sequences, heads, n, 7])
    lens = rng.integers(n // 2, n + 1, sequences)
    lens[0] = n
    if sequences > 2:
        lens[1:3] = 1, 0
    attend_case(kvo, ctx, rng, sequences, 1, heads, n, 1, None, 16, lens=lens)


def test_attend_nan_in_one_split(kvo, ctx):
    """A NaN that one of three CTAs sees reaches the whole result of its query, and no other query's."""
    rng = np.random.default_rng(39)
    n, nq = 400, 45
    rows = random_rows(rng, nq * n)
    rows[3 * n + 350, 512:514] = 0xFF
    cache = kvo.Cache(rows=dev(rows), block_rows=n)
    q = dev(rng.standard_normal((nq, 64, 576)), torch.bfloat16)
    lens = [n] * nq
    out, lse = ctx.attend(cache, q, dev(lens, torch.int32), 0.07, rows=n)
    assert ctx.sync() == kvo.KVO_OK
    assert torch.isnan(lse[3]).all() and torch.isnan(out[3][:, :64]).all()
    keep = [t for t in range(nq) if t != 3][:8]
    check_attend(out[keep], lse[keep], q[keep], 0.07, [list(rows[t * n:(t + 1) * n]) for t in keep], 64)


@pytest.mark.parametrize("heads", [16, 64])
def test_attend_odd_lists(kvo, ctx, heads):
    """Padding entries, repeated ones, entries past the length, in no order; a list with nothing visible."""
    rng = np.random.default_rng(31)
    sel = rng.integers(-3, 400, (4, 200)).astype(np.int32)
    sel[1] = -1
    sel[2] = 7
    sel[3, :] = 2 ** 31 - 1
    sel[3, 150] = 0
    attend_case(kvo, ctx, rng, 4, 1, heads, 300, 1, None, 16, lens=np.array([250, 300, 300, 1]), sel=sel)
    sel[3, :] = (2 ** 31 - 1) // 16
    attend_case(kvo, ctx, rng, 4, 1, heads, 300, 16, None, 16, lens=np.array([250, 300, 113, 0]), sel=sel)


def test_attend_wide_logits(kvo, ctx):
    """Logits of hundreds, growing and falling along the list: the running maximum has to move."""
    rng = np.random.default_rng(32)
    for order in (1, -1):
        n, heads = 1500, 16
        rows = random_rows(rng, n)
        for j in range(n):                                   # rope part grows with the position
            x = np.zeros(64)
            x[:8] = (j if order > 0 else n - j) / 20
            rows[j, 528:] = np.ascontiguousarray(O.bf16_bits(x)).view(np.uint8)
        q = rng.standard_normal((1, heads, 576))
        q[..., 512:520] = np.linspace(-1, 4, heads)[None, :, None]
        q = dev(q, torch.bfloat16)
        cache = kvo.Cache(rows=dev(rows), block_rows=n)
        out, lse = ctx.attend(cache, q, dev([n], torch.int32), 0.5, rows=n)
        assert ctx.sync() == kvo.KVO_OK
        check_attend(out, lse, q, 0.5, [list(rows)], heads)


def test_attend_extreme_scales(kvo, ctx):
    rng = np.random.default_rng(33)
    for scale in (0.0, -0.07, 1e-30):
        attend_case(kvo, ctx, rng, 1, 1, 16, 200, 1, None, 16, scale=scale)
    attend_case(kvo, ctx, rng, 1, 1, 16, 200, 1, None, 16, rows_scale=(6e-8, 6e-7))


@pytest.mark.parametrize("heads", [5, 64])
def test_attend_masked_rows_never_reach_the_output(kvo, ctx, heads):
    """NaN and infinite rows past the length, in unlisted blocks and beside them."""
    rng = np.random.default_rng(34)
    n, br = 400, 16
    table, total = block_table(rng, 1, n // br)
    rows = random_rows(rng, total * br)
    poison = rows.copy()
    lens = 333
    sel = np.sort(rng.choice(n // br, 17, replace=False)).astype(np.int32)[None]
    sel[0, 3] = lens // br
    sel = np.unique(sel)[None]
    seen = set(O.positions_of(sel[0], br, lens, n))
    bad = [O.row_of(table, total, br, 1, 0, p) for p in range(n) if p not in seen]
    bad += [r for r in range(total * br) if r // br not in table]
    poison[bad, 512:] = 0xFF                                  # NaN scales and position parts
    poison[bad[::2], 512:528] = np.array([0x7C00] * 8, np.uint16).view(np.uint8)
    q = dev(rng.standard_normal((1, heads, 576)), torch.bfloat16)
    res = []
    for r in (rows, poison):
        cache = kvo.Cache(rows=dev(r), block_rows=br, table=dev(table))
        res.append(ctx.attend(cache, q, dev([lens], torch.int32), 0.07, sel=dev(sel), sel_block=br))
        assert ctx.sync() == kvo.KVO_OK
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    lists = [[rows[O.row_of(table, total, br, 1, 0, p)] for p in sorted(seen)]]
    check_attend(*res[1], q, 0.07, lists, heads)


def test_attend_visible_nan_shows(kvo, ctx):
    rng = np.random.default_rng(35)
    rows = random_rows(rng, 300)
    rows[200, 512:514] = 0xFF
    cache = kvo.Cache(rows=dev(rows), block_rows=300)
    q = dev(rng.standard_normal((1, 4, 576)), torch.bfloat16)
    out, lse = ctx.attend(cache, q, dev([300], torch.int32), 0.07, rows=300)
    assert ctx.sync() == kvo.KVO_OK
    assert torch.isnan(lse).all() and torch.isnan(out[..., :64]).all()


def test_attend_bad_pages(kvo, ctx):
    rng = np.random.default_rng(36)
    rows = random_rows(rng, 64)
    table = np.array([[1, -1, 3, 0], [2, 0, 77, 9999]], np.int32)
    cache = kvo.Cache(rows=dev(rows), block_rows=16, table=dev(table))
    q = dev(rng.standard_normal((2, 12, 576)), torch.bfloat16)
    for lens, want in (([64, 60], kvo.KVO_ERANGE), ([16, 32], kvo.KVO_OK), ([0, 0], kvo.KVO_OK)):
        out, lse = ctx.attend(cache, q, dev(lens, torch.int32), 0.07, rows=64)
        assert ctx.sync() == want
        lists = []
        for t in range(2):
            at = [O.row_of(table, 4, 16, 2, t, p) for p in range(lens[t])]
            lists.append([rows[r] for r in at if r is not None])
        check_attend(out, lse, q, 0.07, lists, 12)


def test_attend_strided_queries_and_contiguous_rows(kvo, ctx):
    rng = np.random.default_rng(37)
    n, heads = 150, 24
    rows = random_rows(rng, 3 * n)
    wide = dev(rng.standard_normal((3, 2 * heads, 584)), torch.bfloat16)
    q = wide[:, 1::2, 8:]
    cache = kvo.Cache(rows=dev(rows), block_rows=n)
    lens = [150, 149, 3]
    out, lse = ctx.attend(cache, q, dev(lens, torch.int32), 0.07, rows=n)
    assert ctx.sync() == kvo.KVO_OK
    check_attend(out, lse, q, 0.07, [list(rows[t * n:t * n + lens[t]]) for t in range(3)], heads)


def test_attend_no_positions_at_all(kvo, ctx):
    rows = torch.zeros(16, 656, dtype=torch.uint8, device="cuda")
    cache = kvo.Cache(rows=rows, block_rows=16)
    q = torch.randn(2, 20, 576, device="cuda").bfloat16()[:1]
    lens = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    empty = torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    for kw in (dict(rows=0), dict(sel=torch.full((1, 5), -1, dtype=torch.int32, device="cuda")), dict(sel=empty)):
        out, lse = ctx.attend(cache, q, lens, 0.07, **kw)
        assert ctx.sync() == kvo.KVO_OK
        assert not out.any() and torch.isneginf(lse).all()


def test_repeated_calls_give_the_same_bits(kvo, ctx):
    rng = np.random.default_rng(38)
    rows = dev(random_rows(rng, 6000))
    cache = kvo.Cache(rows=rows, block_rows=6000)
    q = dev(rng.standard_normal((1, 64, 576)), torch.bfloat16)
    lens = dev([6000], torch.int32)
    first = ctx.attend(cache, q, lens, 0.07, rows=6000)
    for _ in range(3):
        again = ctx.attend(cache, q, lens, 0.07, rows=6000)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("order", ["rising", "falling", "jumps"])
def test_attend_many_tiles_a_query(kvo, ctx, heads, order):
    """Enough queries that each list stays with one CTA, and logits (in powers of two, up to +-700) that rise, fall or
    jump along it: references move, accumulators are rescaled, early weights vanish."""
    rng = np.random.default_rng([39, heads, len(order)])
    n, nq = 700, 170
    rows = random_rows(rng, n)
    level = {"rising": np.linspace(-40, 40, n), "falling": np.linspace(40, -40, n),
             "jumps": np.where(np.arange(n) // 90 % 3 == 1, 40.0, -40.0) * (np.arange(n) > 200)}[order]
    for j in range(n):
        x = np.zeros(64)
        x[0] = level[j]
        rows[j, 528:] = np.ascontiguousarray(O.bf16_bits(x)).view(np.uint8)
    q = rng.standard_normal((nq, heads, 576))
    q[..., 512] = np.linspace(-12, 12, heads)
    q = dev(q, torch.bfloat16)
    lens = rng.integers(1, n + 1, nq)
    lens[3], lens[77], lens[160] = n, 81, 80
    cache = kvo.Cache(rows=dev(rows), block_rows=n)
    out, lse = ctx.attend(cache, q, dev(lens, torch.int32), 1.0, rows=n)
    assert ctx.sync() == kvo.KVO_OK
    for t in (0, 3, 77, 160, 169):
        check_attend(out[t:t + 1], lse[t:t + 1], q[t:t + 1], 1.0, [list(rows[:lens[t]])], heads)


def test_attend_far_into_a_large_cache(kvo, ctx):
    """Rows whose byte offsets pass 2^31 and 2^32, and whose row numbers differ only there."""
    rng = np.random.default_rng(40)
    total = 7_000_000                                        # 4.6 GB
    rows = torch.zeros(total, 656, dtype=torch.uint8, device="cuda")
    small = random_rows(rng, 64)
    at = np.array([5, 3_300_000, 6_600_000, 6_999_984 // 16 * 16]) // 16
    for b, i in enumerate(at):
        rows[i * 16:(i + 1) * 16] = dev(small[16 * b:16 * b + 16])
    table = torch.tensor(at[None], dtype=torch.int32, device="cuda")
    cache = kvo.Cache(rows=rows, block_rows=16, table=table)
    q = dev(rng.standard_normal((1, 20, 576)), torch.bfloat16)
    out, lse = ctx.attend(cache, q, dev([64], torch.int32), 0.07, rows=64)
    assert ctx.sync() == kvo.KVO_OK
    check_attend(out, lse, q, 0.07, [list(small)], 20)
    kv = dev(rng.standard_normal((1, 576)), torch.bfloat16)
    ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], dev([63], torch.int32), INV_FREQ)
    assert ctx.sync() == kvo.KVO_OK
    got = rows[int(at[3]) * 16 + 15].cpu().numpy()
    for group in range(8):
        want, bits = O.latent_group(f64(kv)[0, 64 * group:64 * group + 64])
        assert np.array_equal(got[64 * group:64 * group + 64].view(np.int8), want)
        assert int(got[512 + 2 * group:514 + 2 * group].view(np.uint16)[0]) == bits


def test_scores_far_into_a_large_cache(kvo, ctx):
    rng = np.random.default_rng(41)
    total = 36_000_000                                       # 4.6 GB of e4m3 keys
    keys = torch.zeros(total, 128, dtype=torch.uint8, device="cuda")
    q, k, scales, w = score_inputs(rng, 1, 16, 64, "e4m3")
    every = torch.zeros(total, device="cuda")
    at = np.array([7, 17_000_000, 34_000_000, total - 16]) // 16
    for b, i in enumerate(at):
        keys[i * 16:(i + 1) * 16] = k.view(torch.uint8)[16 * b:16 * b + 16]
        every[i * 16:(i + 1) * 16] = scales[16 * b:16 * b + 16]
    cache = kvo.Cache(keys=keys.view(torch.float8_e4m3fn), key_scales=every, block_rows=16,
                      table=torch.tensor(at[None], dtype=torch.int32, device="cuda"))
    got = ctx.index_scores(cache, q, w, dev([64], torch.int32), 64)
    assert ctx.sync() == kvo.KVO_OK
    check_scores(got, q, k, scales, w, [list(range(64))], [64], 64, 1)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 100])
def test_scores_tiny_contiguous_caches(kvo, ctx, dtype, n):
    """Caches with fewer keys than a tile, without a table: what lies past them is never looked at."""
    rng = np.random.default_rng([42, n])
    q, k, scales, w = score_inputs(rng, 2, 33, 2 * n, dtype)
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=n)
    got = ctx.index_scores(cache, q, w, dev([n, n], torch.int32), n)
    assert ctx.sync() == kvo.KVO_OK
    check_scores(got, q, k, scales, w, [list(range(n)), list(range(n, 2 * n))], [n, n], n, 1)


def test_strided_tables(kvo, ctx):
    """A table that is a part of a wider one."""
    rng = np.random.default_rng(43)
    wide = torch.full((3, 9), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    table = wide[:, 2:5]
    ids, total = block_table(rng, 3, 3)
    table.copy_(dev(ids))
    rows = random_rows(rng, total * 16)
    q, k, scales, w = score_inputs(rng, 3, 8, total * 16, "e4m3")
    cache = kvo.Cache(rows=dev(rows), keys=k, key_scales=scales, block_rows=16, table=table)
    lens = [48, 20, 33]
    qa = dev(rng.standard_normal((3, 9, 576)), torch.bfloat16)
    out, lse = ctx.attend(cache, qa, dev(lens, torch.int32), 0.07, rows=48)
    got = ctx.index_scores(cache, q, w, dev(lens, torch.int32), 48)
    assert ctx.sync() == kvo.KVO_OK
    where = [[O.row_of(ids, total, 16, 3, s, p) for p in range(48)] for s in range(3)]
    check_attend(out, lse, qa, 0.07, [[rows[r] for r in where[s][:lens[s]]] for s in range(3)], 9)
    check_scores(got, q, k, scales, w, where, lens, 48, 1)


def test_binding_refuses_wrong_shapes(kvo, ctx):
    rows = torch.zeros(32, 656, dtype=torch.uint8, device="cuda")
    cache = kvo.Cache(rows=rows, block_rows=16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.zeros(2, 4, 576, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[:, :, :512]), dict(q=q[:1]), dict(q=q.transpose(1, 2)), dict(lens=i32(3)),
                dict(lens=i32(2).long()), dict(rows=None), dict(sel=i32(2)), dict(sel=i32(3, 4)),
                dict(out=torch.zeros(2, 4, 512, device="cuda")), dict(lse=torch.zeros(2, 5, device="cuda")),
                dict(out=torch.zeros(2, 512, 4, dtype=torch.bfloat16, device="cuda").transpose(1, 2))):
        with pytest.raises(ValueError):
            ctx.attend(cache, **{**dict(q=q, lens=i32(2), scale=0.1, rows=16), **bad})
    with pytest.raises(ValueError):
        ctx.index_scores(cache, q[..., :128], torch.zeros(2, 4, device="cuda"), i32(2), 16)
    kv = torch.zeros(2, 576, device="cuda")
    for bad in (dict(latent=kv[:, :500]), dict(latent=kv[:, :512].double()), dict(rope=kv[:, 512:].bfloat16()),
                dict(pos=i32(3)), dict(inv_freq=INV_FREQ[:8]), dict(seq=i32(2).long()), dict(latent=kv[:, :512].cpu())):
        with pytest.raises(ValueError):
            ctx.append_tokens(cache, **{**dict(latent=kv[:, :512], rope=kv[:, 512:], pos=i32(2), inv_freq=INV_FREQ),
                                        **bad})
    with pytest.raises(kvo.KvoError):                        # no keys in the cache
        ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], i32(2), INV_FREQ, key=torch.zeros(2, 128, device="cuda"))
    assert ctx.sync() == kvo.KVO_OK


# ------------------------------------------------------------- streams, graphs
def decode_step(kvo, ctx, st, stream=None):
    ctx.append_tokens(st["cache"], st["kv"][:, :512], st["kv"][:, 512:], st["pos"], INV_FREQ, key=st["key"],
                      stream=stream)
    ctx.index_scores(st["cache"], st["qi"], st["w"], st["lens"], st["n"], out=st["scores"], stream=stream)
    ctx.select_topk_batch(st["scores"], st["k"], idx=st["idx"], stream=stream)
    return ctx.attend(st["cache"], st["q"], st["lens"], 0.07, sel=st["idx"], out=st["out"], lse=st["lse"],
                      work=st["work"], stream=stream)


def decode_state(kvo, seed, S=3, n=400, k=96, heads=20):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    blocks = -(-n // 16)
    table = torch.randperm(S * blocks, generator=g, device="cuda").int().view(S, blocks)
    rows = torch.zeros(S * blocks * 16, 656, dtype=torch.uint8, device="cuda")
    keys = torch.zeros(S * blocks * 16, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    st = dict(cache=kvo.Cache(rows=rows, keys=keys, key_scales=torch.zeros(S * blocks * 16, device="cuda"),
                              block_rows=16, table=table),
              kv=rand(S, 576).bfloat16(), key=rand(S, 128).bfloat16(),
              qi=rand(S, 32, 128).to(torch.float8_e4m3fn), w=rand(S, 32), q=rand(S, heads, 576).bfloat16(),
              pos=torch.full((S,), n - 1, dtype=torch.int32, device="cuda"),
              lens=torch.full((S,), n, dtype=torch.int32, device="cuda"), n=n, k=k,
              scores=torch.empty(S, n, device="cuda"), idx=torch.empty(S, k, dtype=torch.int32, device="cuda"),
              out=torch.empty(S, heads, 512, dtype=torch.bfloat16, device="cuda"),
              lse=torch.empty(S, heads, device="cuda"), rows=rows)
    need = kvo.kvo_attend_work_bytes(S, heads, k)
    st["work"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return st, rand


def prefill(kvo, ctx, st, rand):
    S, n = st["lens"].numel(), st["n"]
    kv, key = rand(S * n, 576).bfloat16(), rand(S * n, 128).bfloat16()
    seq = torch.arange(S, device="cuda").repeat_interleave(n).int()
    pos = torch.arange(n, device="cuda").repeat(S).int()
    ctx.append_tokens(st["cache"], kv[:, :512], kv[:, 512:], pos, INV_FREQ, seq=seq, key=key)


def test_side_stream_and_graph_give_the_same_bits(kvo, ctx):
    st, rand = decode_state(kvo, 41)
    prefill(kvo, ctx, st, rand)
    decode_step(kvo, ctx, st)
    assert ctx.sync() == kvo.KVO_OK
    want = [st[k].clone() for k in ("rows", "scores", "idx", "out", "lse")]
    side = torch.cuda.Stream()

    def same():
        return all(torch.equal(a, st[k]) for a, k in zip(want, ("rows", "scores", "idx", "out", "lse")))

    def spoil():
        for k in ("scores", "idx", "out", "lse"):
            st[k].zero_()
        st["work"].fill_(0xFF)
        torch.cuda.synchronize()

    spoil()
    decode_step(kvo, ctx, st, stream=side)
    side.synchronize()
    assert same()
    spoil()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode_step(kvo, ctx, st)
    for _ in range(2):
        spoil()
        graph.replay()
        torch.cuda.synchronize()
        assert same()
    assert ctx.sync() == kvo.KVO_OK


def test_outputs_made_on_a_given_stream(kvo, ctx):
    """Outputs and scratch that a call makes itself belong to the stream it is given."""
    st, rand = decode_state(kvo, 42, n=3000, k=2048)
    prefill(kvo, ctx, st, rand)
    decode_step(kvo, ctx, st)
    assert ctx.sync() == kvo.KVO_OK
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        out, lse = ctx.attend(st["cache"], st["q"], st["lens"], 0.07, sel=st["idx"], stream=side)
        scores = ctx.index_scores(st["cache"], st["qi"], st["w"], st["lens"], st["n"], stream=side)
    side.synchronize()
    assert torch.equal(out, st["out"]) and torch.equal(lse, st["lse"]) and torch.equal(scores, st["scores"])


@pytest.mark.parametrize("captured", [False, True])
def test_inputs_written_just_before_and_spoilt_just_after(kvo, ctx, captured):
    """Every call's launch may be scheduled while the work before it runs: it reads nothing that slow kernels on its
    own stream and on another that it waits for have yet to write, and kernels behind it change nothing for it."""
    st, rand = decode_state(kvo, 43, n=1000, k=512, heads=64)
    prefill(kvo, ctx, st, rand)
    decode_step(kvo, ctx, st)
    assert ctx.sync() == kvo.KVO_OK
    results = ("rows", "scores", "idx", "out", "lse")
    want = {k: st[k].clone() for k in results}
    inputs = {"append": (("kv", "key"), ("pos",)), "score": (("qi", "w"), ("lens",)), "attend": (("q",), ("lens",))}
    good = {k: st[k].clone() for own, other in inputs.values() for k in own + other}
    bad = {k: torch.full_like(v.float(), -5.0 if k in ("pos", "lens") else float("nan")).to(v.dtype) for k, v in good.items()}
    load = torch.randn(32 << 20, device="cuda")
    side = torch.cuda.Stream()

    def spoil(names):
        for k in names:
            st[k].copy_(bad[k])

    def step(main):
        def call(name):
            own, other = inputs[name]
            side.wait_stream(main)
            for stream, names in ((side, other), (main, own)):
                with torch.cuda.stream(stream):
                    load.mul_(1.0)
                    for k in names:
                        st[k].copy_(good[k])
            main.wait_stream(side)
            with torch.cuda.stream(main):
                if name == "append":
                    ctx.append_tokens(st["cache"], st["kv"][:, :512], st["kv"][:, 512:], st["pos"], INV_FREQ,
                                      key=st["key"])
                elif name == "score":
                    ctx.index_scores(st["cache"], st["qi"], st["w"], st["lens"], st["n"], out=st["scores"])
                    ctx.select_topk_batch(st["scores"], st["k"], idx=st["idx"])
                else:
                    ctx.attend(st["cache"], st["q"], st["lens"], 0.07, sel=st["idx"], out=st["out"], lse=st["lse"],
                               work=st["work"])
                spoil(own + other)

        for name in inputs:
            call(name)

    main = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    spoil(good)
    torch.cuda.synchronize()
    if captured:
        with torch.cuda.graph(graph, stream=main):
            step(torch.cuda.current_stream())
    for _ in range(3):
        for k in results[1:]:
            st[k].zero_()
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            step(main)
        torch.cuda.synchronize()
        assert all(torch.equal(want[k], st[k]) for k in results)
    assert ctx.sync() == kvo.KVO_OK


def test_two_streams_at_once(kvo, ctx):
    """Steps of two independent states on two streams, interleaved: neither changes the other's bits."""
    states, want, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed, (n, k, heads) in enumerate([(3000, 2048, 64), (700, 96, 20)]):
        st, rand = decode_state(kvo, 60 + seed, S=2 + seed, n=n, k=k, heads=heads)
        prefill(kvo, ctx, st, rand)
        decode_step(kvo, ctx, st)
        states.append(st)
    assert ctx.sync() == kvo.KVO_OK
    names = ("rows", "scores", "idx", "out", "lse")
    for st in states:
        want.append([st[k].clone() for k in names])
        for k in names[1:]:
            st[k].zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for st, stream in zip(states, streams):
            decode_step(kvo, ctx, st, stream=stream)
    torch.cuda.synchronize()
    for st, w in zip(states, want):
        assert all(torch.equal(a, st[k]) for a, k in zip(w, names))
    assert ctx.sync() == kvo.KVO_OK


# ----------------------------------------------------------- with the rest
def test_gathered_rows_attend_like_the_pool(kvo):
    """append -> history -> one decode step's gathered rows -> attend gives what attending in place gives."""
    n, k, heads = 600, 128, 16
    c = kvo.Context(1, n, 256)
    g = torch.Generator(device="cuda")
    g.manual_seed(51)
    kv = torch.randn(n, 576, generator=g, device="cuda").bfloat16()
    rows = torch.zeros(n, 656, dtype=torch.uint8, device="cuda")
    flat = kvo.Cache(rows=rows, block_rows=n)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    values = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
    c.append_tokens(flat, kv[:, :512], kv[:, 512:], pos, INV_FREQ, seq=torch.zeros_like(pos), out_bf16=values)
    c.append_rows(0, rows)
    scores = torch.randn(n, generator=g, device="cuda")
    idx = torch.empty(k, dtype=torch.int32, device="cuda")
    got = torch.empty(k, 656, dtype=torch.uint8, device="cuda")
    deq = torch.empty(k, 576, dtype=torch.bfloat16, device="cuda")
    c.decode_layers([dict(layer=0, scores=scores, idx=idx, out_rows=got, out_bf16=deq)], k)
    q = torch.randn(1, heads, 576, generator=g, device="cuda").bfloat16()
    a = c.attend(kvo.Cache(rows=got, block_rows=k), q, torch.full((1,), k, dtype=torch.int32, device="cuda"), 0.07, rows=k)
    b = c.attend(flat, q, torch.full((1,), n, dtype=torch.int32, device="cuda"), 0.07, sel=idx[None])
    assert c.sync() == kvo.KVO_OK
    assert torch.equal(deq, values[idx.long()])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_attend(*a, q, 0.07, [list(got.cpu().numpy())], heads)
    c.close()


def test_pool_session_rows(kvo, ctx):
    """Rows appended into a session's pool blocks are what the pool's own calls read back."""
    pool = kvo.Pool(layers=2, pool_blocks=20, block_tokens=16, tier_blocks=0)
    assert pool.alloc(5, 50) == kvo.KVO_OK
    table = torch.tensor([kvo.kvo_pool_block_table(pool.handle, 5, 1)], dtype=torch.int32, device="cuda")
    cache = kvo.Cache(rows=pool, table=table)
    assert cache.block_rows == 16 and cache.blocks == 20
    kv = torch.randn(50, 576, device="cuda").bfloat16()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], pos, INV_FREQ, seq=torch.zeros_like(pos))
    flat = torch.zeros(50, 656, dtype=torch.uint8, device="cuda")
    ctx.append_tokens(kvo.Cache(rows=flat, block_rows=50), kv[:, :512], kv[:, 512:], pos, INV_FREQ,
                      seq=torch.zeros_like(pos))
    back = torch.empty(50, 656, dtype=torch.uint8, device="cuda")
    pool.read(5, 1, 0, back)
    assert ctx.sync() == kvo.KVO_OK
    assert torch.equal(back, flat)
    pool.close()


@pytest.mark.parametrize("block", [1, 16])
def test_example(block):
    """The example's decode: with k past the context the selection is everything, and holds the whole softmax."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_decode.py")
    spec = importlib.util.spec_from_file_location("sparse_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.decode(sessions=2, prompt=300, steps=3, k=4_096 if block > 1 else 303, block=block)
    # log-sum-exps of the same rows in another order: within the bound of their sums
    assert (r["lse"] - r["all_lse"]).abs().max() < 1e-4 and abs(r["share"] - 1) < 1e-4
    assert torch.isfinite(r["out"].float()).all()
    some = example.decode(sessions=2, prompt=300, steps=2, k=64, block=block)
    assert 0 < some["share"] < 1 and (some["lse"] < some["all_lse"]).all()
    assert some["idx"].shape == (2, 64 // block) and (some["idx"].diff(dim=1) > 0).all()


def test_an_unusable_context_refuses(kvo):
    """After a wait whose copies may still land, nothing more is launched."""
    c = kvo.Context(1, 64, 64)
    c.raise_status(4 | 8)
    assert c.sync() == kvo.KVO_ETIMEDOUT
    rows = torch.zeros(16, 656, dtype=torch.uint8, device="cuda")
    keys = torch.zeros(16, 128, dtype=torch.bfloat16, device="cuda")
    cache = kvo.Cache(rows=rows, keys=keys, block_rows=16)
    lens = torch.full((1,), 16, dtype=torch.int32, device="cuda")
    kv = torch.zeros(1, 576, device="cuda").bfloat16()
    for call in (lambda: c.append_tokens(cache, kv[:, :512], kv[:, 512:], lens - 1, INV_FREQ),
                 lambda: c.index_scores(cache, kv[None, :, :128], torch.zeros(1, 1, device="cuda"), lens, 16),
                 lambda: c.attend(cache, kv[None], lens, 0.1, rows=16)):
        with pytest.raises(kvo.KvoError) as e:
            call()
        assert e.value.status == kvo.KVO_ECUDA
    torch.cuda.synchronize()
    assert not rows.any()
    c.close()


def test_a_closed_pool_is_refused(kvo, ctx):
    pool = kvo.Pool(layers=1, pool_blocks=2, block_tokens=16, tier_blocks=0)
    cache = kvo.Cache(rows=pool)
    pool.close()
    with pytest.raises(ValueError):
        ctx.attend(cache, torch.zeros(2, 1, 576, dtype=torch.bfloat16, device="cuda"),
                   torch.ones(2, dtype=torch.int32, device="cuda"), 0.1, rows=16)


@pytest.mark.parametrize("block_rows", [1, 16])
def test_a_table_without_columns_has_no_rows(kvo, ctx, block_rows):
    """Every position is masked and says so: nothing is written to, or read from, the block of the sequence's number."""
    rng = np.random.default_rng(51)
    held = dev(random_rows(rng, 4 * block_rows))
    keys = dev(rng.standard_normal((4 * block_rows, 128)), torch.bfloat16)
    rows_before, keys_before = held.clone(), keys.clone()
    cache = kvo.Cache(rows=held, keys=keys, block_rows=block_rows, table=torch.empty(2, 0, dtype=torch.int32, device="cuda"))
    kv = dev(rng.standard_normal((2, 576)), torch.bfloat16)
    values = torch.full((2, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], lens - 1, INV_FREQ, key=kv[:, :128], out_bf16=values)
    assert ctx.sync() == kvo.KVO_ERANGE
    assert torch.equal(held, rows_before) and torch.equal(keys, keys_before) and not values.any()
    scores = ctx.index_scores(cache, kv[:, None, :128], torch.ones(2, 1, device="cuda"), lens, 3)
    assert ctx.sync() == kvo.KVO_ERANGE and torch.isneginf(scores).all()
    out, lse = ctx.attend(cache, kv[:, None], lens, 0.1, rows=1)
    assert ctx.sync() == kvo.KVO_ERANGE and not out.any() and torch.isneginf(lse).all()
    scores = ctx.index_scores(cache, kv[:, None, :128], torch.ones(2, 1, device="cuda"), lens - 1, 3)
    assert ctx.sync() == kvo.KVO_OK and torch.isneginf(scores).all()      # nothing visible: no entry is needed


@pytest.mark.parametrize("heads", [1, 8, 24, 32, 40, 64, 100, 128])
@pytest.mark.parametrize("per_seq,block", [(1, 1), (1, 16), (3, 1), (2, 4)])
def test_scores_infinite_keys(kvo, ctx, heads, per_seq, block):
    """An infinite key scores the sum over the heads there are, whatever they are rounded up to: 0 where every
    product is -inf, +inf where one is +inf, NaN where infinities of both signs meet."""
    rng = np.random.default_rng([52, heads, per_seq, block])
    n = 400
    q, k, _, w = score_inputs(rng, per_seq, heads, n, "bf16")
    signs = dev(rng.choice([-1.0, 1.0], (per_seq, heads)), torch.bfloat16)
    q[:, :, 3], q[:, :, 4], q[:, :, 5] = 1.5, -0.75, signs          # the dimensions that infinite keys have
    w = w.abs() + 0.125
    w[-1] *= dev(rng.choice([-1.0, 1.0], heads), torch.float32)     # the last token's weights of both signs
    infinite = {5: (3, math.inf), 70: (4, math.inf), 131: (5, math.inf), 140: (3, -math.inf), 290: (4, -math.inf),
                399: (5, -math.inf)}
    for at, (d, x) in infinite.items():
        k[at, d] = x
    cache = kvo.Cache(keys=k, block_rows=n)
    got = f64(ctx.index_scores(cache, q, w, torch.full((per_seq,), n, dtype=torch.int32, device="cuda"), n, block=block))
    assert ctx.sync() == kvo.KVO_OK
    rows, lens = [list(range(n))] * per_seq, [n] * per_seq
    want, _ = O.index_scores(f64(q), f64(w), f64(k), np.ones(n), rows, lens, block)
    clean = f64(k)
    clean[~np.isfinite(clean)] = 0.0                                # what is finite at an infinite key is exactly 0
    _, size = O.index_scores(f64(q), f64(w), clean, np.ones(n), rows, lens, block)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    assert (np.abs(got[fin] - want[fin]) <= ((128 + heads + 2) * 2 * U * size)[fin]).all()
    assert per_seq == 1 or np.isposinf(want[0]).any()
    assert block > 1 or (want[:, 70] == 0).all()


# Waits that run out.  Clocks of 0 say that a wait has given up before the first one; a few clocks end some waits or
# none, as the GPU's work falls: a call then ends in KVO_ETIMEDOUT, or gives what it always gives.
WAITS = (0, 0, 1, 100, 1_000, 4_000, 0, 20_000, 400)


def check_waits(kvo, run):
    """`run(context)` returns outputs; nothing of a call that timed out is in the next one's way."""
    c = kvo.Context(1, 64, 64)
    want = [t.clone() for t in run(c)]
    assert c.sync() == kvo.KVO_OK
    for clocks in WAITS:
        c.set_wait_clocks(clocks)
        got = run(c)
        status = c.sync()
        assert status in ((kvo.KVO_ETIMEDOUT,) if clocks == 0 else (kvo.KVO_OK, kvo.KVO_ETIMEDOUT))
        assert c.sync() == kvo.KVO_OK                            # said once, and the context goes on
        c.set_wait_clocks()
        for again in (got if status == kvo.KVO_OK else None, run(c)):
            for a, b in zip(again or (), want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), clocks
        assert c.sync() == kvo.KVO_OK
    c.close()


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("sequences,per_seq,heads,n,block,block_rows", [
    (1, 1, 16, 100, 1, 16), (1, 1, 64, 160_000, 1, 16), (1, 4, 64, 60_000, 128, 0), (1, 2, 20, 30_000, 4, 5),
    (120, 1, 64, 1_500, 1, 16), (90, 5, 64, 700, 64, 48)])
def test_scores_waits_that_run_out(kvo, dtype, sequences, per_seq, heads, n, block, block_rows):
    rng = np.random.default_rng([53, sequences, per_seq, heads, n])
    nq = sequences * per_seq
    br = block_rows or n
    blocks = -(-n // br)
    total = sequences * blocks
    q, k, scales, w = score_inputs(rng, nq, heads, total * br, dtype)
    table = None if not block_rows else dev(rng.permutation(total).reshape(sequences, blocks).astype(np.int32))
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=br, table=table)
    lens = dev(rng.integers(0, n + 1, nq), torch.int32)
    lens[0] = n
    check_waits(kvo, lambda c: [c.index_scores(cache, q, w, lens, n, block=block)])


@pytest.mark.parametrize("sequences,heads,n,sel_block,picked,block_rows", [
    (1, 64, 70, 1, None, 16), (1, 16, 40_000, 1, None, 16), (2, 64, 30_000, 1, None, 64), (1, 128, 20_000, 1, 2048, 16),
    (160, 64, 600, 1, None, 16), (170, 20, 900, 16, 30, 16), (77, 40, 2_000, 1, 700, 48)])
def test_attend_waits_that_run_out(kvo, sequences, heads, n, sel_block, picked, block_rows):
    rng = np.random.default_rng([54, sequences, heads, n, sel_block])
    blocks, total = -(-n // block_rows), max(4_000 // block_rows, 8)
    table = dev(rng.integers(0, total, (sequences, blocks)).astype(np.int32))
    cache = kvo.Cache(rows=dev(random_rows(rng, total * block_rows)), block_rows=block_rows, table=table)
    q = dev(rng.standard_normal((sequences, heads, 576)), torch.bfloat16)
    lens = dev(rng.integers(0, n + 1, sequences), torch.int32)
    lens[0] = n
    sel = None
    if picked is not None:
        sel = dev(np.sort(rng.integers(0, n // sel_block, (sequences, picked)), 1).astype(np.int32))
    check_waits(kvo, lambda c: c.attend(cache, q, lens, 192 ** -0.5, rows=n, sel=sel, sel_block=sel_block))


@pytest.mark.parametrize("interleaved", [True, False])
def test_append_negative_frequencies(kvo, ctx, interleaved):
    """Rotations backwards, of small frequencies among them, up to position 2^31 - 1."""
    rng = np.random.default_rng(55)
    freq = -INV_FREQ
    freq[::3] = -np.exp(rng.uniform(np.log(1e-19), np.log(1e-7), len(freq[::3])))
    pos = np.array([0, 1, 4_097, 1_048_575, 2 ** 31 - 1], np.int32)
    n, block = len(pos), 2 ** 30
    rows = torch.zeros(n, 656, dtype=torch.uint8, device="cuda")
    kv = rng.standard_normal((n, 576)).astype(np.float32)
    for i, p in enumerate(pos):
        # one block of 2^30 rows, of which only the addressed row exists: its base is shifted
        table = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
        table[0, int(p) // block] = 0
        big = kvo.Cache(rows=rows[i:i + 1], block_rows=1, table=table)
        big.c.block_rows, big.c.blocks = block, 1
        big.c.rows = rows.data_ptr() + i * 656 - (int(p) % block) * 656
        ctx.append_tokens(big, dev(kv[i:i + 1, :512]), dev(kv[i:i + 1, 512:]), dev(pos[i:i + 1]), freq,
                          interleaved=interleaved)
    assert ctx.sync() == kvo.KVO_OK
    out = rows.cpu().numpy()
    for i, p in enumerate(pos):
        x = kv[i, 512:].astype(np.float64)
        exact = O.rotate(x, int(p), freq, interleaved)
        pair = np.abs(x[0::2]) + np.abs(x[1::2]) if interleaved else np.abs(x[:32]) + np.abs(x[32:])
        pair = np.repeat(pair, 2) if interleaved else np.tile(pair, 2)
        assert (np.abs(O.row_values(out[i])[1] - exact) <= 2.0 ** -8 * np.abs(exact) + 8 * U * pair).all(), p


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lengths", ["uneven", "one long", "none"])
@pytest.mark.parametrize("sequences,per_seq,heads,n,block,block_rows", [
    (80, 4, 24, 500, 64, 48), (310, 1, 5, 2_000, 2, 48), (100, 3, 32, 700, 128, 64), (90, 2, 128, 400, 8, 5)])
def test_scores_tiles_shared_out(kvo, ctx, dtype, lengths, sequences, per_seq, heads, n, block, block_rows):
    """More than half as many tasks as SMs, few tiles each: several tokens in 128 and 256 columns, blocks beyond a warp."""
    test_scores_many_sequences(kvo, ctx, dtype, lengths, sequences, per_seq, heads, n, block, block_rows)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("per_seq,heads,n,block,block_rows", [
    (1, 16, 170_003, 1, 16), (4, 64, 130_000, 1, 0), (2, 40, 150_001, 16, 5), (1, 64, 260_000, 64, 64)])
def test_scores_of_long_contexts(kvo, ctx, dtype, per_seq, heads, n, block, block_rows):
    """One row of the grid a sequence, and many more tiles a CTA than its ring has slots and its accumulators."""
    rng = np.random.default_rng([56, per_seq, heads, n])
    br = block_rows or n
    blocks = -(-n // br)
    q, k, scales, w = score_inputs(rng, per_seq, heads, blocks * br, dtype)
    order = rng.permutation(blocks)
    table = dev(order[None].astype(np.int32)) if block_rows else None
    lens = np.array([n - 17 * g for g in range(per_seq)])
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=br, table=table)
    got = f64(ctx.index_scores(cache, q, w, dev(lens, torch.int32), n, block=block))
    assert ctx.sync() == kvo.KVO_OK
    at = np.arange(n)
    rows = order[at // br] * br + at % br if block_rows else at
    keys, factors = f64(k)[rows], np.ones(n) if scales is None else f64(scales)[rows]
    for g in range(per_seq):
        qg, wg = f64(q[g]), f64(w[g])
        want = factors * (np.maximum(keys @ qg.T, 0.0) @ wg)
        size = factors * ((np.abs(keys) @ np.abs(qg).T) @ np.abs(wg))
        want[lens[g]:], size[lens[g]:] = -np.inf, 0.0
        pad = -n % block
        want = np.pad(want, (0, pad), constant_values=-np.inf).reshape(-1, block).max(1)
        size = np.pad(size, (0, pad)).reshape(-1, block).max(1)
        fin = np.isfinite(want)
        assert np.array_equal(np.isfinite(got[g]), fin)
        assert (np.abs(got[g][fin] - want[fin]) <= ((128 + heads + 2) * 2 * U * size)[fin]).all()


@pytest.mark.parametrize("dtype,sequences,per_seq,heads,n", [("e4m3", 1, 300, 32, 700), ("bf16", 2, 131, 64, 300),
                                                             ("e4m3", 3, 65, 7, 200)])
def test_scores_of_a_prompt(kvo, ctx, dtype, sequences, per_seq, heads, n):
    """Every token of a prompt sees those up to its own."""
    rng = np.random.default_rng([57, sequences, per_seq, heads, n])
    nq, br = sequences * per_seq, 16
    blocks = -(-n // br)
    table, total = block_table(rng, sequences, blocks)
    q, k, scales, w = score_inputs(rng, nq, heads, total * br, dtype)
    lens = np.tile(n - per_seq + 1 + np.arange(per_seq), sequences)
    cache = kvo.Cache(keys=k, key_scales=scales, block_rows=br, table=dev(table))
    got = ctx.index_scores(cache, q, w, dev(lens, torch.int32), n)
    assert ctx.sync() == kvo.KVO_OK
    assert np.array_equal(np.isneginf(f64(got)), np.arange(n)[None] >= lens[:, None])
    some = np.unique(np.concatenate([rng.choice(nq, 40, replace=False), [0, per_seq - 1, nq - 1]]))
    rows = [[O.row_of(table, total, br, sequences, t // per_seq, p) for p in range(n)] for t in some]
    check_scores(got[some], q[some], k, scales, w[some], rows, lens[some], n, 1)


@pytest.mark.parametrize("sequences,per_seq,heads", [(1, 200, 8), (2, 90, 20), (1, 170, 64)])
@pytest.mark.parametrize("listed", [False, True])
def test_attend_of_a_prompt(kvo, ctx, sequences, per_seq, heads, listed):
    rng = np.random.default_rng([58, sequences, per_seq, heads, int(listed)])
    n = per_seq + 40
    lens = np.tile(41 + np.arange(per_seq), sequences)
    attend_case(kvo, ctx, rng, sequences, per_seq, heads, n, 1, 50 if listed else None, 16, lens=lens)


@pytest.mark.parametrize("sequences,heads", [(76, 64), (77, 64), (100, 33), (152, 16), (153, 64), (77, 128)])
@pytest.mark.parametrize("listed", [False, True])
def test_attend_batches_about_the_number_of_sms(kvo, ctx, sequences, heads, listed):
    """Batches on either side of half, of all, and of twice the SMs of this GPU."""
    rng = np.random.default_rng([59, sequences, heads, int(listed)])
    attend_case(kvo, ctx, rng, sequences, 1, heads, 260, 1, 150 if listed else None, 16)


@pytest.mark.parametrize("dtype,key,interleaved", [("bf16", "e4m3", True), ("fp16", "bf16", False), ("fp32", "e4m3", False)])
def test_append_prompt_pieces(kvo, ctx, dtype, key, interleaved):
    """Runs of several sequences' next positions, over many CTAs and a partly filled last one."""
    rng = np.random.default_rng([60, len(dtype), len(key)])
    n, sequences, br = 603, 5, 64
    seqs = np.sort(rng.integers(0, sequences, n)).astype(np.int32)
    first = np.searchsorted(seqs, np.arange(sequences))
    pos = (np.arange(n) - first[seqs] + 7 * seqs).astype(np.int32)
    assert pos.max() < 3 * br
    r = append_case(kvo, ctx, rng, dtype, n, interleaved, key, br, seqs=seqs, pos=pos, sequences=sequences)
    assert r["status"] == kvo.KVO_OK
    # pairs that hold an infinity (fp16 inputs overflow) are compared as what they are, and as zeros from there on
    for i, j in zip(*np.nonzero(~np.isfinite(r["kv"][:, 512:576]))):
        at = O.row_of(r["table"], r["blocks"], br, sequences, int(seqs[i]), int(pos[i]))
        pair = [j // 2 * 2, j // 2 * 2 + 1] if interleaved else [j % 32, j % 32 + 32]
        with np.errstate(invalid="ignore"):
            exact = O.rotate(r["kv"][i, 512:576], int(pos[i]), INV_FREQ, interleaved)[pair]
        bits = r["rows"][at, 528:].view(np.uint16)
        assert not np.isfinite(exact).any() and np.array_equal(O.row_values(r["rows"][at])[1][pair], exact, equal_nan=True)
        assert np.array_equal(f64(r["values"])[i, 512:][pair], exact, equal_nan=True)
        bits[pair] = 0
        r["values"][i, 512 + np.array(pair)] = 0
        r["kv"][i, 512 + np.array(pair)] = 0.0
    check_append(kvo, r, dtype, interleaved, key, br)


@pytest.mark.parametrize("heads,n", [(5, 40), (64, 300), (20, 9_000)])
def test_attend_infinite_logits(kvo, ctx, heads, n):
    """-inf weighs nothing, and all of them leave an empty query; +inf is a NaN, in its own heads alone."""
    rng = np.random.default_rng([61, heads, n])
    rows = random_rows(rng, 3 * n)
    rope = rows[:, 528:].view(np.uint16)
    rope[:n, 7] = O.bf16_bits([-math.inf])[0]                       # sequence 0: every row
    rope[n:2 * n:3, 7] = O.bf16_bits([-math.inf])[0]                # 1: every third
    rope[2 * n + n // 2, 7] = O.bf16_bits([math.inf])[0]            # 2: one, above
    q = rng.standard_normal((3, heads, 576))
    q[:, :, 519] = 1.0
    q[2, 1::2, 519] = -1.0                                          # -inf there for every other head
    q = dev(q, torch.bfloat16)
    cache = kvo.Cache(rows=dev(rows), block_rows=n)
    out, lse = ctx.attend(cache, q, torch.full((3,), n, dtype=torch.int32, device="cuda"), 192 ** -0.5, rows=n)
    assert ctx.sync() == kvo.KVO_OK
    assert not out[0].any() and torch.isneginf(lse[0]).all()
    left = [[], [rows[n + i] for i in range(n) if i % 3], [rows[2 * n + i] for i in range(n) if i != n // 2]]
    check_attend(out[1:2], lse[1:2], q[1:2], 192 ** -0.5, left[1:2], heads)
    assert torch.isnan(out[2, 0::2]).all() and torch.isnan(lse[2, 0::2]).all()
    check_attend(out[2:, 1::2], lse[2:, 1::2], q[2:, 1::2], 192 ** -0.5, left[2:], heads // 2)
