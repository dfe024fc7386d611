"""kvo_attend_chunk, kvo_attention_weights and kvo_shrink_cache against the 64-bit oracle.

Tolerances, from the number formats alone (u = 2^-24, half a step of fp32; 2^-8, half a step of bf16):
  lse      the logits' error (576 steps of 2 u of the magnitudes: an accumulator may truncate), the exponentials and the
           logarithm 16 u, a blocked sum 2 u for each of n / 128 + 32 steps, and 2 u of its size;
  out      2^-8 |out| for its rounding, and for the sum of p |v| the weights' rounding 2^-8, twice the logits' error and
           the steps of the sum as above.
           Weights are held down to 2^-94 of the largest (2^-126 below a reference up to 2^32 above it), and a smaller
           one takes at most 2^-94 |v| with it: 2^-80 for 2^13 positions of latents below 2;
  weights  every term p = exp(z - lse) off by p times the error of its logit, 4 u of |lse| (its product with log2 e and
           the difference, each rounded) and 16 u for the exponential; the sum of a tile's 128 terms and the carried
           tiles 64 u of its size; and 2 u of keep * carry.
What is chosen and copied has to be equal.
"""
import numpy as np
import pytest
import torch

from oracle import kvo_chunk_oracle as C
from oracle import kvo_sparse_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SCALE = 192 ** -0.5


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


class Chunk:
    """Queries of a ragged batch over a paged cache, and what the calls on them have to give."""

    def __init__(self, kvo, rng, counts, lens, heads, block_rows=16, rows=None, scale=SCALE, gain=1.0, q=None, raw=None,
                 table=None, first=0, after=0):
        self.kvo, self.counts, self.lens, self.heads, self.scale = kvo, counts, list(lens), heads, scale
        self.n, self.rows = len(counts), max(max(lens), 0) if rows is None else rows
        self.starts = first + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.tokens = int(self.starts[-1]) + after
        br = self.br = block_rows or max(self.rows, 1)
        if block_rows:
            self.table, self.total = block_table(rng, self.n, max(1, -(-self.rows // br)))
        else:
            self.table, self.total = None, self.n
        if table is not None:
            self.table, self.total = table
        self.raw = random_rows(rng, self.total * br) if raw is None else raw
        self.q = dev(rng.standard_normal((self.tokens, heads, 576)) * gain, torch.bfloat16) if q is None else q
        self.cache = kvo.Cache(rows=dev(self.raw), block_rows=br, table=None if self.table is None else dev(self.table),
                               sequences=self.n if self.table is None else None)
        self.dev_starts, self.dev_lens = dev(self.starts), dev(self.lens, torch.int32)

    def keys(self, s, n):
        """Values of the sequence's first n positions that have a row, and their positions."""
        at = [O.row_of(self.table, self.total, self.br, self.n, s, p) for p in range(n)]
        have = [p for p, r in enumerate(at) if r is not None]
        return C.values([self.raw[at[p]] for p in have]), np.array(have, int)

    def attend(self, ctx, **kw):
        return ctx.attend_chunk(self.cache, self.q, self.dev_starts, self.dev_lens, self.scale, self.rows, **kw)

    def check_attend(self, out, lse):
        out, lse, q = f64(out), f64(lse), f64(self.q)
        for s in range(self.n):
            keys, have = self.keys(s, min(max(self.lens[s], 0), self.rows))
            for t in C.tokens_of(self.starts, s):
                n = int((have < C.seen(self.starts, self.lens, s, t, self.rows)).sum())
                want, want_lse, spread, size = C.attend(q[t], self.scale, keys[:n])
                if n == 0:
                    assert not out[t].any() and np.isneginf(lse[t]).all(), (s, t)
                    continue
                steps, logit = n / 128 + 32, 2 * U * 576 * size
                tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2 * logit + 16 * U + 2 * U * steps)[:, None]
                tol += 2.0 ** -80
                assert (np.abs(out[t] - want) <= tol).all(), (s, t, float((np.abs(out[t] - want) / tol).max()))
                tol = logit + 16 * U + 2 * U * steps + 2 * U * np.abs(want_lse)
                assert (np.abs(lse[t] - want_lse) <= tol).all(), (s, t, float((np.abs(lse[t] - want_lse) / tol).max()))

    def lse(self):
        """The log-sum-exps as attention returns them."""
        q, out = f64(self.q), np.full((self.tokens, self.heads), -np.inf)
        for s in range(self.n):
            keys, have = self.keys(s, min(max(self.lens[s], 0), self.rows))
            for t in C.tokens_of(self.starts, s):
                n = int((have < C.seen(self.starts, self.lens, s, t, self.rows)).sum())
                out[t] = C.attend(q[t], self.scale, keys[:n])[1]
        return dev(out, torch.float32)

    def weights(self, ctx, lse, **kw):
        return ctx.attention_weights(self.cache, self.q, self.dev_starts, self.dev_lens, lse, self.scale, self.rows, **kw)

    def check_weights(self, got, lse, window=0, carry=None, keep=1.0):
        got, lse, q = f64(got), f64(lse), f64(self.q)
        assert got.shape == (self.n, self.rows)
        for s in range(self.n):
            held = min(max(self.lens[s], 0), self.rows)
            keys, have = self.keys(s, held)
            want, tol = np.zeros(self.rows), np.full(self.rows, 2.0 ** -120)
            if carry is not None:
                want[:held] = keep * f64(carry)[s, :held]
                tol += 4 * U * np.abs(want)
            tokens = list(C.tokens_of(self.starts, s))
            for t in tokens[-window:] if window else tokens:
                n = int((have < C.seen(self.starts, self.lens, s, t, self.rows)).sum())
                add, share = C.weights(q[t], self.scale, keys[:n], lse[t])
                want[have[:n]] += add
                tol[have[:n]] += (2 * 576 + 4) * U * share + (16 + 64) * U * add
            assert (np.abs(got[s] - want) <= tol).all(), (s, float((np.abs(got[s] - want) / tol).max()))


# ------------------------------------------------------------------ attention
SHAPES = [
    ([1], [1], 1, 1), ([1], [61], 16, 0), ([1], [300], 128, 16), ([4], [4], 16, 16), ([7], [500], 20, 48),
    ([1, 4, 2], [70, 33, 129], 64, 16), ([33], [257], 5, 7), ([130], [130], 16, 16), ([5, 0, 40, 1], [900, 77, 41, 640], 24, 64),
    ([64], [4000], 8, 16), ([3] * 40, list(range(3, 123, 3)), 16, 16), ([2], [1500], 100, 16)]


@pytest.mark.parametrize("counts,lens,heads,block_rows", SHAPES)
def test_chunk(kvo, ctx, counts, lens, heads, block_rows):
    rng = np.random.default_rng([71, sum(counts), max(lens), heads])
    c = Chunk(kvo, rng, counts, lens, heads, block_rows)
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)


@pytest.mark.parametrize("heads", [3, 16, 64])
def test_chunk_tokens_that_see_nothing(kvo, ctx, heads):
    """Fewer positions than tokens, none, a negative length; `rows` below a length."""
    rng = np.random.default_rng([72, heads])
    c = Chunk(kvo, rng, [9, 20, 5, 6, 0], [4, 0, -7, 200, 90], heads, rows=150)
    c.lens[0] = 4
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    c = Chunk(kvo, rng, [9, 20], [0, 0], heads, rows=0)
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("counts,lens,heads", [([6, 0, 3], [200, 10, 33], 20), ([40], [5000], 64), ([3], [40], 128)])
def test_chunk_leaves_other_tokens_alone(kvo, ctx, counts, lens, heads):
    """Tokens before the first sequence's and behind the last one's."""
    rng = np.random.default_rng([73, heads])
    c = Chunk(kvo, rng, counts, lens, heads, first=2, after=5)
    out = torch.full((c.tokens, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.tokens, heads), 7.0, device="cuda")
    c.attend(ctx, out=out, lse=lse)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    for x in (out, lse):
        assert (x[:2] == 7).all() and (x[-5:] == 7).all()


@pytest.mark.parametrize("order", ["rising", "falling", "one"])
@pytest.mark.parametrize("tokens,heads", [(1, 16), (9, 20), (300, 16)])
def test_chunk_wide_logits(kvo, ctx, order, tokens, heads):
    """Logits of hundreds that rise or fall along the positions, or one position far above all others."""
    rng = np.random.default_rng([74, tokens, heads, len(order)])
    n = 1300
    raw = random_rows(rng, n)
    for j in range(n):
        x = np.zeros(64)
        x[:8] = {"rising": j / 20, "falling": (n - j) / 20, "one": 60.0 * (j == 777)}[order]
        raw[j, 528:] = np.ascontiguousarray(O.bf16_bits(x)).view(np.uint8)
    q = rng.standard_normal((tokens, heads, 576))
    q[..., 512:520] = np.linspace(-1, 4, heads)[None, :, None]
    c = Chunk(kvo, rng, [tokens], [n], heads, 0, scale=0.5, q=dev(q, torch.bfloat16), raw=raw)
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)


@pytest.mark.parametrize("heads,tokens", [(5, 12), (16, 40), (64, 40), (64, 300)])
def test_chunk_values_that_are_not_seen(kvo, ctx, heads, tokens):
    """A row that reads as NaN: the tokens before it give what they give without it, the others are NaN.  Rows past the
    length, whatever they hold, change nothing."""
    rng = np.random.default_rng([75, heads, tokens])
    n, at = 333, 333 - tokens // 2
    c = Chunk(kvo, rng, [tokens], [n], heads, rows=400)
    clean = c.attend(ctx)
    raw = c.raw.copy()
    past = [O.row_of(c.table, c.total, 16, 1, 0, p) for p in range(n, 400)]
    raw[past, 512:] = 0xFF
    nan = O.row_of(c.table, c.total, 16, 1, 0, at)
    for kind in range(3):
        spoilt = raw.copy()
        if kind == 0:
            spoilt[nan, 518:520] = 0xFF                       # a NaN scale
        elif kind == 1:
            spoilt[nan, 512:514] = np.array([0x7C00], np.uint16).view(np.uint8)   # an infinite one
        else:
            spoilt[nan, 600:602] = 0xFF                       # a NaN in the position part
        d = Chunk(kvo, rng, [tokens], [n], heads, rows=400, q=c.q, raw=spoilt, table=(c.table, c.total))
        out, lse = d.attend(ctx)
        assert ctx.sync() == kvo.KVO_OK
        before = at - (n - tokens)                            # tokens that do not see it
        assert torch.equal(out[:before], clean[0][:before]) and torch.equal(lse[:before], clean[1][:before])
        assert torch.isnan(lse[before:]).all() and torch.isnan(out[before:, :, :64]).all()


@pytest.mark.parametrize("tokens", [4, 200])
def test_chunk_infinite_logits(kvo, ctx, tokens):
    """Position parts that make logits -inf for some heads: nothing from them, and nothing at all from only such."""
    rng = np.random.default_rng([76, tokens])
    n, heads = 260, 20
    raw = random_rows(rng, n)
    raw[3::7, 528:530] = np.array([0x7F80], np.uint16).view(np.uint8)             # +inf
    q = np.abs(rng.standard_normal((tokens, heads, 576)))
    q[:, :, 512] = -np.abs(q[:, :, 512])
    c = Chunk(kvo, rng, [tokens], [n], heads, 0, q=dev(q, torch.bfloat16), raw=raw)
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    gone = [p for p in range(n) if p % 7 == 3]
    keys = C.values(raw)
    for t in range(tokens):
        seen = C.seen(c.starts, c.lens, 0, t, n)
        have = [p for p in range(seen) if p not in gone]
        want, want_lse, spread, size = C.attend(f64(c.q)[t], SCALE, keys[have])
        tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 4 * U * 576 * size + 100 * U)[:, None]
        assert (np.abs(f64(out)[t] - want) <= tol).all()
        assert (np.abs(f64(lse)[t] - want_lse) <= 2 * U * 576 * size + 100 * U + 2 * U * np.abs(want_lse)).all()
    raw[:, 528:530] = np.array([0x7F80], np.uint16).view(np.uint8)
    c = Chunk(kvo, rng, [tokens], [n], heads, 0, q=c.q, raw=raw)
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("heads,tokens", [(12, 3), (64, 50), (128, 200)])
def test_chunk_bad_pages(kvo, ctx, heads, tokens):
    """Entries without a block mask what they would hold, at the front too, and say so only when they are needed."""
    rng = np.random.default_rng([77, heads])
    table = np.array([[-1, 1, -5, 3, 0, 77, 2 ** 31 - 1], [2, 0, 77, 9999, -1, -1, -1]], np.int32)
    for lens, want in (([112, 60], kvo.KVO_ERANGE), ([80, 20], kvo.KVO_ERANGE), ([0, 32], kvo.KVO_OK)):
        c = Chunk(kvo, rng, [tokens, min(tokens, 7)], lens, heads, 16, rows=112, table=(table, 4))
        out, lse = c.attend(ctx)
        assert ctx.sync() == want
        c.check_attend(out, lse)


def test_chunk_bad_starts(kvo, ctx):
    """Starts outside the tokens, or that go back: an error is latched, and nothing behind the outputs is touched."""
    rng = np.random.default_rng(78)
    c = Chunk(kvo, rng, [4, 4, 4], [100, 90, 80], 20)
    for starts in ([0, 4, 8, 13], [-1, 4, 8, 12], [0, 9, 4, 12], [0, 4, 2 ** 31 - 1, 12], [0, -2 ** 31, 8, 12]):
        wide = torch.full((14, 20, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(12, 20, device="cuda")
        bad = dev(starts, torch.int32)
        ctx.attend_chunk(c.cache, c.q, bad, c.dev_lens, SCALE, 100, out=wide[1:13], lse=lse)
        assert ctx.sync() == kvo.KVO_ERANGE, starts
        assert (wide[0] == 7).all() and (wide[13] == 7).all()
        ctx.attention_weights(c.cache, c.q, bad, c.dev_lens, lse, SCALE, 100)
        assert ctx.sync() == kvo.KVO_ERANGE, starts


@pytest.mark.parametrize("counts,lens,heads", [([3, 2], [90, 41], 24), ([70], [300], 16), ([5], [200], 128), ([40, 41], [99, 200], 7)])
def test_chunk_strides(kvo, ctx, counts, lens, heads):
    """Queries as views of wider ones, and heads before tokens."""
    rng = np.random.default_rng([79, heads])
    c = Chunk(kvo, rng, counts, lens, heads)
    want, want_lse = c.attend(ctx)
    c.check_attend(want, want_lse)
    weights = c.weights(ctx, want_lse)
    wide = torch.full((c.tokens, 2 * heads, 592), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1::2, 8:584] = c.q
    across = torch.empty(heads, c.tokens, 576, dtype=torch.bfloat16, device="cuda")
    across.copy_(c.q.transpose(0, 1))
    for q in (wide[:, 1::2, 8:584], across.transpose(0, 1)):
        c.q = q
        out, lse = c.attend(ctx)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        got = c.weights(ctx, want_lse)
        assert ctx.sync() == kvo.KVO_OK
        c.check_weights(got, want_lse)
    del weights


def test_chunk_of_one_token_is_attend(kvo, ctx):
    """The decode form: a token a sequence gives what kvo_attend gives, to the rounding of both."""
    rng = np.random.default_rng(80)
    c = Chunk(kvo, rng, [1] * 5, [300, 1, 0, 77, 160], 20)
    out, lse = c.attend(ctx)
    one, one_lse = ctx.attend(c.cache, c.q, c.dev_lens, SCALE, rows=300)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    c.check_attend(one, one_lse)


# -------------------------------------------------------------------- weights
@pytest.mark.parametrize("counts,lens,heads,block_rows", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 3])
def test_weights(kvo, ctx, counts, lens, heads, block_rows, window):
    rng = np.random.default_rng([81, sum(counts), max(lens), heads])
    c = Chunk(kvo, rng, counts, lens, heads, block_rows)
    lse = c.lse()
    carry = dev(rng.exponential(1.0, (c.n, c.rows)), torch.float32)
    got = c.weights(ctx, lse, window=window, carry=carry, keep=0.875)
    assert ctx.sync() == kvo.KVO_OK
    c.check_weights(got, lse, window, carry, 0.875)


@pytest.mark.parametrize("counts,lens,heads", [([700], [900], 16), ([300], [300], 64), ([64, 1, 200], [2500, 513, 255], 20)])
def test_weights_of_many_tokens(kvo, ctx, counts, lens, heads):
    """Several tiles of columns, in one pair of CTAs and split; what a token gives adds up to one a head."""
    rng = np.random.default_rng([82, sum(counts), heads])
    c = Chunk(kvo, rng, counts, lens, heads)
    out, lse = c.attend(ctx)
    got = c.weights(ctx, lse)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    c.check_weights(got, lse)
    total = got.double().sum(1).cpu().numpy()
    assert np.allclose(total, np.array(counts) * heads, rtol=1e-4)


def test_weights_edges(kvo, ctx):
    """Tokens that see nothing, sequences without tokens or positions, strides, in place, and -inf from a masked lse."""
    rng = np.random.default_rng(83)
    c = Chunk(kvo, rng, [9, 20, 0, 6, 2], [4, 0, 40, 200, -5], 24, rows=170)
    lse = c.lse()
    wide = dev(rng.exponential(1.0, (5, 400)), torch.float32)
    carry = wide[:, 7:177].clone()
    got = c.weights(ctx, lse, carry=wide[:, 7:177], keep=0.5, out=wide[:, 7:177])
    assert ctx.sync() == kvo.KVO_OK
    c.check_weights(got, lse, 0, carry, 0.5)
    lse[29:33, 3:9] = -float("inf")
    got = c.weights(ctx, lse)
    assert ctx.sync() == kvo.KVO_OK
    c.check_weights(got, lse)
    none = Chunk(kvo, rng, [0, 0], [50, 3], 8)
    carry = dev(rng.exponential(1.0, (2, 50)), torch.float32)
    got = none.weights(ctx, torch.empty(0, 8, device="cuda"), carry=carry)
    assert ctx.sync() == kvo.KVO_OK
    assert torch.equal(got[0], carry[0]) and torch.equal(got[1, :3], carry[1, :3]) and not got[1, 3:].any()


def test_weights_are_not_reached_by_hidden_values(kvo, ctx):
    """NaN rows past the length, NaN queries of a neighbouring sequence, a NaN row that only later tokens see."""
    rng = np.random.default_rng(84)
    c = Chunk(kvo, rng, [3, 5, 4], [150, 90, 33], 20, rows=160)
    lse = c.lse()
    clean = c.weights(ctx, lse)
    c.check_weights(clean, lse)
    raw = c.raw.copy()
    for s in range(3):
        for p in range(c.lens[s], 160):
            raw[O.row_of(c.table, c.total, 16, 3, s, p), 512:] = 0xFF
    q = c.q.clone()
    q[8:] = float("nan")
    d = Chunk(kvo, rng, [3, 5, 4], [150, 90, 33], 20, rows=160, q=q, raw=raw, table=(c.table, c.total))
    got = d.weights(ctx, lse)
    assert ctx.sync() == kvo.KVO_OK
    assert torch.equal(got[:2], clean[:2]) and torch.isnan(got[2, :30]).all()
    raw = c.raw.copy()
    raw[O.row_of(c.table, c.total, 16, 3, 1, 87), 528:530] = 0xFF
    d = Chunk(kvo, rng, [3, 5, 4], [150, 90, 33], 20, rows=160, q=c.q, raw=raw, table=(c.table, c.total))
    got = d.weights(ctx, lse)
    assert torch.isnan(got[1, 87])
    got[1, 87] = clean[1, 87]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("counts,lens", [([3, 2], [112, 60]), ([30, 30], [80, 64])])
def test_weights_bad_pages(kvo, ctx, counts, lens):
    rng = np.random.default_rng(85)
    table = np.array([[-1, 1, -5, 3, 0, 77, 2 ** 31 - 1], [2, 0, 77, 9999, -1, -1, -1]], np.int32)
    c = Chunk(kvo, rng, counts, lens, 12, 16, rows=112, table=(table, 4))
    lse = c.lse()
    carry = dev(rng.exponential(1.0, (2, 112)), torch.float32)
    got = c.weights(ctx, lse, carry=carry)
    assert ctx.sync() == kvo.KVO_ERANGE
    c.check_weights(got, lse, 0, carry)


# --------------------------------------------------------------------- shrink
def shrink_case(kvo, ctx, rng, lens, n, budget, first, last, key, block_rows, to_rows=None, weights=None, strided=False):
    sequences = len(lens)
    br, to_br = block_rows or n, to_rows or block_rows or budget
    table, total = block_table(rng, sequences, -(-n // br)) if block_rows else (None, sequences)
    to_table, to_total = block_table(rng, sequences, -(-budget // to_br)) if block_rows or to_rows else (None, sequences)
    raw = random_rows(rng, total * br)
    src, dst = dict(rows=dev(raw)), dict(rows=torch.full((to_total * to_br, 656), 0x5A, dtype=torch.uint8, device="cuda"))
    if key != "none":
        keys = dev(rng.integers(0, 255, (total * br, 128 if key == "e4m3" else 256), dtype=np.uint8))
        kind = torch.float8_e4m3fn if key == "e4m3" else torch.bfloat16
        src["keys"] = keys.view(kind)
        dst["keys"] = torch.full((to_total * to_br, keys.shape[1]), 0x22, dtype=torch.uint8, device="cuda").view(kind)
        if key == "e4m3":
            src["key_scales"] = dev(rng.exponential(1.0, total * br), torch.float32)
            dst["key_scales"] = torch.full((to_total * to_br,), 5.0, device="cuda")
    if weights is None:
        weights = rng.exponential(1.0, (sequences, n)).astype(np.float32)
        weights[rng.random((sequences, n)) < 0.3] = 0.0
    a = kvo.Cache(**src, block_rows=br, table=None if table is None else dev(table))
    b = kvo.Cache(**dst, block_rows=to_br, table=None if to_table is None else dev(to_table))
    w, kw = dev(weights), {}
    if strided:
        wide = torch.full((sequences, n + 9), float("nan"), device="cuda")
        wide[:, 4:n + 4] = w
        w = wide[:, 4:n + 4]
        kw = dict(kept=torch.full((sequences, budget + 3), 77, dtype=torch.int32, device="cuda")[:, 1:budget + 1],
                  to_weights=torch.full((sequences, budget + 5), 77.0, device="cuda")[:, 2:budget + 2])
    kept, new_lens, to_weights = ctx.shrink_cache(a, b, w, dev(lens, torch.int32), budget, first, last, **kw)
    assert ctx.sync() == kvo.KVO_OK
    want_rows = np.full((to_total * to_br, 656), 0x5A, np.uint8)
    want_keys = None if key == "none" else np.full((to_total * to_br, src["keys"].view(torch.uint8).shape[1]), 0x22, np.uint8)
    want_scales = np.full(to_total * to_br, 5.0, np.float32)
    for s, have in enumerate(lens):
        have = min(max(have, 0), n)
        stay = C.keep(weights[s], have, budget, first, last)
        assert int(new_lens[s]) == len(stay)
        assert kept[s].tolist() == stay + [-1] * (budget - len(stay)), s
        got = to_weights[s].cpu().numpy()
        assert np.array_equal(got[:len(stay)], weights[s, stay], equal_nan=True) and not got[len(stay):].any()
        for j, p in enumerate(stay):
            x = O.row_of(table, total, br, sequences, s, p)
            y = O.row_of(to_table, to_total, to_br, sequences, s, j)
            want_rows[y] = raw[x]
            if key != "none":
                want_keys[y] = src["keys"][x].view(torch.uint8).cpu().numpy()
            if key == "e4m3":
                want_scales[y] = float(src["key_scales"][x])
    assert np.array_equal(dst["rows"].cpu().numpy(), want_rows)
    if key != "none":
        assert np.array_equal(dst["keys"].view(torch.uint8).cpu().numpy(), want_keys)
    if key == "e4m3":
        assert np.array_equal(dst["key_scales"].cpu().numpy(), want_scales)
    if strided:
        assert (kw["kept"]._base[:, 0] == 77).all() and (kw["kept"]._base[:, budget + 1:] == 77).all()
        assert (kw["to_weights"]._base[:, :2] == 77).all() and (kw["to_weights"]._base[:, budget + 2:] == 77).all()


@pytest.mark.parametrize("key", ["none", "bf16", "e4m3"])
@pytest.mark.parametrize("lens,n,budget,first,last,block_rows", [
    ([1], 1, 1, 0, 0, 1), ([50], 50, 1, 0, 1, 16), ([300], 300, 77, 4, 10, 16), ([300, 0, 77, 78, -3, 500], 300, 77, 0, 77, 48),
    ([90, 41, 64], 90, 64, 64, 0, 7), ([700], 700, 699, 1, 1, 0), ([64] * 20, 64, 33, 1, 2, 16)])
def test_shrink(kvo, ctx, key, lens, n, budget, first, last, block_rows):
    rng = np.random.default_rng([91, n, budget, len(lens)])
    shrink_case(kvo, ctx, rng, lens, n, budget, first, last, key, block_rows)
    shrink_case(kvo, ctx, rng, lens, n, budget, first, last, key, block_rows, to_rows=5, strided=True)


@pytest.mark.parametrize("kind", ["ties", "specials", "falling", "negative"])
@pytest.mark.parametrize("n,budget", [(100, 37), (9000, 4100), (9000, 8999)])
def test_shrink_orders(kvo, ctx, kind, n, budget):
    """Equal weights, infinities, NaN and zeros of both signs at the border."""
    rng = np.random.default_rng([92, n, budget, len(kind)])
    w = {"ties": rng.integers(0, 3, (2, n)).astype(np.float32),
         "specials": rng.choice(np.array([0.0, -0.0, np.nan, -np.nan, np.inf, -np.inf, 1e-45, -1e-45, 1.0], np.float32), (2, n)),
         "falling": np.tile(np.linspace(1, 0, n, dtype=np.float32), (2, 1)),
         "negative": -rng.exponential(1.0, (2, n)).astype(np.float32)}[kind]
    shrink_case(kvo, ctx, rng, [n, n - 50], n, budget, 2, 3, "none", 16, weights=w)


@pytest.mark.parametrize("n,budget,sequences", [(70_001, 20_000, 1), (30_000, 1_000, 9), (900_000, 450_001, 1), (2_500, 300, 200)])
def test_shrink_large(kvo, ctx, n, budget, sequences):
    """Clusters of every width, keys in shared memory and not; compared on the GPU with a stable sort."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    lens = torch.full((sequences,), n, dtype=torch.int32, device="cuda")
    lens[sequences // 2:] -= 7
    w = torch.rand(sequences, n, generator=g, device="cuda")
    w = torch.where(w < 0.6, (w * 50).round(), w)            # many equal ones
    rows = torch.randint(0, 256, (sequences * n, 656), generator=g, dtype=torch.uint8, device="cuda")
    out = torch.zeros(sequences * budget, 656, dtype=torch.uint8, device="cuda")
    a, b = kvo.Cache(rows=rows, block_rows=n), kvo.Cache(rows=out, block_rows=budget)
    kept, new_lens, to_weights = ctx.shrink_cache(a, b, w, lens, budget, first=5, last=100)
    assert ctx.sync() == kvo.KVO_OK
    assert (new_lens == budget).all()
    for s in range(sequences):
        have = int(lens[s])
        order = w[s, :have].clone()
        order[:5] = order[have - 100:] = 1e9
        want = order.sort(descending=True, stable=True).indices[:budget].sort().values
        assert torch.equal(kept[s].long(), want)
        assert torch.equal(to_weights[s], w[s, want])
        assert torch.equal(out[s * budget:(s + 1) * budget], rows[s * n + want])


def test_shrink_bad_pages(kvo, ctx):
    """A source without a row becomes zeros, a destination without one is dropped; both are said."""
    rng = np.random.default_rng(94)
    raw = random_rows(rng, 64)
    table = np.array([[1, -1, 3, 0], [2, 0, 77, 9999]], np.int32)
    to_table = np.array([[0, 1], [-1, 2]], np.int32)
    w = rng.exponential(1.0, (2, 64)).astype(np.float32)
    out = torch.full((48, 656), 0x5A, dtype=torch.uint8, device="cuda")
    keys = dev(rng.integers(0, 255, (64, 256), dtype=np.uint8)).view(torch.bfloat16)
    to_keys = torch.full((48, 256), 0x5A, dtype=torch.uint8, device="cuda").view(torch.bfloat16)
    a = kvo.Cache(rows=dev(raw), keys=keys, block_rows=16, table=dev(table))
    b = kvo.Cache(rows=out, keys=to_keys, block_rows=16, table=dev(to_table))
    kept, new_lens, _ = ctx.shrink_cache(a, b, dev(w), dev([64, 60], torch.int32), 30, 0, 5)
    assert ctx.sync() == kvo.KVO_ERANGE
    want, want_keys = np.full((48, 656), 0x5A, np.uint8), np.full((48, 256), 0x5A, np.uint8)
    for s in range(2):
        stay = C.keep(w[s], (64, 60)[s], 30, 0, 5)
        assert kept[s].tolist() == stay
        for j, p in enumerate(stay):
            x, y = O.row_of(table, 4, 16, 2, s, p), O.row_of(to_table, 3, 16, 2, s, j)
            if y is not None:
                want[y] = 0 if x is None else raw[x]
                want_keys[y] = 0 if x is None else keys[x].view(torch.uint8).cpu().numpy()
    assert np.array_equal(out.cpu().numpy(), want)
    assert np.array_equal(to_keys.view(torch.uint8).cpu().numpy(), want_keys)


# ------------------------------------------------------------------- together
def session(kvo, ctx, seed, stream=None, sizes=((120, 90), (60, 61)), heads=20, budget=70):
    """Two chunks of two sessions, their attention and weights, then the shrunk cache and a decode step on it."""
    rng = np.random.default_rng(seed)
    n = max(sum(s[i] for s in sizes) for i in range(2))
    br = 16
    table, total = block_table(rng, 2, -(-n // br))
    to_table, to_total = block_table(rng, 2, -(-(budget + 1) // br))
    st = dict(rng=rng, raw=torch.zeros(total * br, 656, dtype=torch.uint8, device="cuda"), table=table, to_table=to_table,
              to=torch.zeros(to_total * br, 656, dtype=torch.uint8, device="cuda"), n=n, heads=heads, budget=budget, br=br)
    st["cache"] = kvo.Cache(rows=st["raw"], block_rows=br, table=dev(table))
    st["small"] = kvo.Cache(rows=st["to"], block_rows=br, table=dev(to_table))
    st["total"], st["to_total"] = total, to_total
    held = np.zeros(2, int)
    st["pieces"] = []
    for piece in sizes:
        seq = np.repeat([0, 1], piece).astype(np.int32)
        pos = np.concatenate([held[s] + np.arange(piece[s]) for s in range(2)]).astype(np.int32)
        held = held + piece
        st["pieces"].append(dict(seq=dev(seq), pos=dev(pos), starts=dev(np.array([0, piece[0], sum(piece)], np.int32)),
                                 lens=dev(held.astype(np.int32)), host=held.copy(),
                                 kv=dev(rng.standard_normal((sum(piece), 576)), torch.bfloat16),
                                 q=dev(rng.standard_normal((sum(piece), heads, 576)), torch.bfloat16)))
    st["weights"] = torch.zeros(2, n, device="cuda")
    st["one"] = dev(rng.standard_normal((2, heads, 576)), torch.bfloat16)
    st["one_kv"] = dev(rng.standard_normal((2, 576)), torch.bfloat16)
    st["one_starts"] = dev(np.arange(3), torch.int32)
    return st


FREQ = 10_000.0 ** (-np.arange(0, 64, 2) / 64)


def run_session(ctx, st, stream=None):
    outs = []
    st["weights"].zero_()
    for p in st["pieces"]:
        ctx.append_tokens(st["cache"], p["kv"][:, :512], p["kv"][:, 512:], p["pos"], FREQ, seq=p["seq"], stream=stream)
        out, lse = ctx.attend_chunk(st["cache"], p["q"], p["starts"], p["lens"], SCALE, st["n"], stream=stream)
        ctx.attention_weights(st["cache"], p["q"], p["starts"], p["lens"], lse, SCALE, st["n"], window=16,
                              carry=st["weights"], keep=0.75, out=st["weights"], stream=stream)
        outs += [out, lse]
    kept, lens, w = ctx.shrink_cache(st["cache"], st["small"], st["weights"], st["pieces"][-1]["lens"], st["budget"], 2, 8,
                                     stream=stream)
    # the next token goes behind what stayed, turned by its own position
    pos = st["pieces"][-1]["lens"]
    at = st["one_kv"]
    ctx.append_tokens(st["small"], at[:, :512], at[:, 512:], lens, FREQ, stream=stream)
    more = lens + 1
    out, lse = ctx.attend_chunk(st["small"], st["one"], st["one_starts"], more, SCALE, st["budget"] + 1, stream=stream)
    del pos
    return outs + [kept, lens, w, st["weights"], out, lse, st["to"], st["raw"]]


def test_a_session_together(kvo, ctx):
    st = session(kvo, ctx, 95)
    outs = run_session(ctx, st)
    assert ctx.sync() == kvo.KVO_OK
    rng = np.random.default_rng(1)
    raw = st["raw"].cpu().numpy()
    mass = None
    for i, p in enumerate(st["pieces"]):
        counts = np.diff(p["starts"].cpu().numpy()).tolist()
        c = Chunk(kvo, rng, counts, p["host"].tolist(), st["heads"], st["br"], rows=st["n"], q=p["q"], raw=raw,
                  table=(st["table"], st["total"]))
        c.check_attend(outs[2 * i], outs[2 * i + 1])
        got = c.weights(ctx, outs[2 * i + 1], window=16, carry=mass, keep=0.75)
        c.check_weights(got, outs[2 * i + 1], 16, mass, 0.75)
        mass = got
    kept, lens, w, total, out, lse = outs[4:10]
    assert torch.equal(mass, total)
    for s in range(2):
        stay = C.keep(total[s].cpu().numpy(), int(st["pieces"][-1]["host"][s]), st["budget"], 2, 8)
        assert kept[s].tolist() == stay and torch.equal(w[s], total[s, stay])
    small = Chunk(kvo, rng, [1, 1], (lens.cpu().numpy() + 1).tolist(), st["heads"], st["br"], rows=st["budget"] + 1,
                  q=st["one"], raw=st["to"].cpu().numpy(), table=(st["to_table"], st["to_total"]))
    small.check_attend(out, lse)


def test_side_stream_graph_and_two_streams(kvo, ctx):
    """The same bits on another stream, captured and replayed on new inputs, and from two sessions at once."""
    a, b = session(kvo, ctx, 96), session(kvo, ctx, 97, sizes=((33, 200), (10, 7)), heads=64, budget=90)
    want = [[t.clone() for t in run_session(ctx, x)] for x in (a, b)]
    assert ctx.sync() == kvo.KVO_OK
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for x in (a, b):
            x["raw"].zero_()
            x["to"].zero_()
        torch.cuda.synchronize()
        got = [None, None]
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = run_session(ctx, x)
        torch.cuda.synchronize()
        for x, y in zip(want[0] + want[1], got[0] + got[1]):
            assert torch.equal(x, y)
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = run_session(ctx, x)
        graphs.append((g, res))
    for p in a["pieces"]:
        p["q"].copy_(p["q"].roll(1, 0))
        p["kv"].copy_(p["kv"].roll(1, 0))
    want[0] = [t.clone() for t in run_session(ctx, a)]
    torch.cuda.synchronize()
    for _ in range(2):
        for i, (g, _) in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                g.replay()
        torch.cuda.synchronize()
        for i, (_, res) in enumerate(graphs):
            for x, y in zip(want[i], res):
                assert torch.equal(x, y)
    assert ctx.sync() == kvo.KVO_OK


WAITS = (0, 0, 1, 100, 1_000, 4_000, 0, 20_000, 400)


@pytest.mark.parametrize("counts,lens,heads", [([3, 2], [300, 40], 20), ([512], [600], 16), ([90, 300], [4000, 900], 64)])
def test_waits_that_run_out(kvo, counts, lens, heads):
    rng = np.random.default_rng([98, sum(counts)])
    c = kvo.Context(1, 64, 64)
    chunk = Chunk(kvo, rng, counts, lens, heads)

    def run(lse=None):
        out, l = chunk.attend(c)
        return out, l, chunk.weights(c, l if lse is None else lse)

    want = [t.clone() for t in run()]
    assert c.sync() == kvo.KVO_OK
    for clocks in WAITS:
        c.set_wait_clocks(clocks)
        got = run(want[1])
        status = c.sync()
        assert status in ((kvo.KVO_ETIMEDOUT,) if clocks == 0 else (kvo.KVO_OK, kvo.KVO_ETIMEDOUT))
        assert c.sync() == kvo.KVO_OK                            # said once, and the context goes on
        c.set_wait_clocks()
        for again in (got if status == kvo.KVO_OK else None, run()):
            for a, b in zip(again or (), want):
                assert torch.equal(a, b), clocks
        assert c.sync() == kvo.KVO_OK
    c.close()


# ------------------------------------------- attention of many tokens at once
class Long(Chunk):
    """The same held positions in a cache with room for many more: enough work for the kernel of many columns."""

    def attend(self, ctx, rows=60_000, **kw):
        blocks = -(-rows // self.br)
        table = np.full((self.n, blocks), -1, np.int32)
        part = np.arange(self.n, dtype=np.int32)[:, None] if self.table is None else self.table[:, :blocks]
        table[:, :part.shape[1]] = part
        cache = self.kvo.Cache(rows=dev(self.raw), block_rows=self.br, table=dev(table))
        return ctx.attend_chunk(cache, self.q, self.dev_starts, self.dev_lens, self.scale, rows, **kw)


@pytest.mark.parametrize("counts,lens,heads,block_rows", [
    ([4], [4], 64, 16), ([4], [300], 64, 16), ([256], [256], 1, 64), ([200], [777], 3, 7), ([13], [1000], 20, 0),
    ([2, 0, 5, 9], [700, 40, 5, 300], 100, 16), ([90], [400], 128, 64), ([64] * 3, [2000, 777, 513], 64, 16),
    ([130, 1, 66], [130, 1, 255], 128, 16), ([33] * 9, [256 * i + 33 for i in range(9)], 16, 64), ([40], [5000], 128, 16)])
def test_long_chunk(kvo, ctx, counts, lens, heads, block_rows):
    rng = np.random.default_rng([101, sum(counts), max(lens), heads])
    c = Long(kvo, rng, counts, lens, heads, block_rows)
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)


@pytest.mark.parametrize("heads", [40, 64, 128])
def test_long_chunk_leaves_other_tokens_alone(kvo, ctx, heads):
    """Tokens before the first sequence's and behind the last one's, tokens that see nothing, negative lengths."""
    rng = np.random.default_rng([102, heads])
    c = Long(kvo, rng, [9, 20, 5, 26, 0], [4, 0, -7, 200, 90], heads, first=2, after=5)
    out = torch.full((c.tokens, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.tokens, heads), 7.0, device="cuda")
    c.attend(ctx, out=out, lse=lse)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    for x in (out, lse):
        assert (x[:2] == 7).all() and (x[-5:] == 7).all()


@pytest.mark.parametrize("order", ["rising", "falling", "one", "steps"])
@pytest.mark.parametrize("n", [200, 1300])
@pytest.mark.parametrize("tokens,heads", [(14, 20), (90, 64)])
def test_long_chunk_wide_logits(kvo, ctx, order, n, tokens, heads):
    """Logits of hundreds along the positions: far above the first tile's for some heads, far below for others."""
    rng = np.random.default_rng([103, tokens, n, len(order)])
    raw = random_rows(rng, n)
    for j in range(n):
        x = np.zeros(64)
        x[:8] = {"rising": j / 20, "falling": (n - j) / 20, "one": 60.0 * (j == n * 3 // 5), "steps": 9.0 * (j // 129)}[order]
        raw[j, 528:] = np.ascontiguousarray(O.bf16_bits(x)).view(np.uint8)
    q = rng.standard_normal((tokens, heads, 576))
    q[..., 512:520] = np.linspace(-1, 4, heads)[None, :, None]
    c = Long(kvo, rng, [tokens], [n], heads, 0, scale=0.5, q=dev(q, torch.bfloat16), raw=raw)
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)


@pytest.mark.parametrize("heads,tokens", [(16, 40), (64, 140)])
def test_long_chunk_values_that_are_not_seen(kvo, ctx, heads, tokens):
    rng = np.random.default_rng([104, heads, tokens])
    n, at = 333, 333 - tokens // 2
    c = Long(kvo, rng, [tokens], [n], heads, rows=400)
    clean = c.attend(ctx)
    raw = c.raw.copy()
    raw[[O.row_of(c.table, c.total, 16, 1, 0, p) for p in range(n, 400)], 512:] = 0xFF
    nan = O.row_of(c.table, c.total, 16, 1, 0, at)
    for kind in range(4):
        spoilt = raw.copy()
        if kind == 0:
            spoilt[nan, 518:520] = 0xFF                       # a NaN scale
        elif kind == 1:
            spoilt[nan, 512:514] = np.array([0x7C00], np.uint16).view(np.uint8)   # an infinite one
        elif kind == 2:
            spoilt[nan, 600:602] = 0xFF                       # a NaN in the position part
        d = Long(kvo, rng, [tokens], [n], heads, rows=400, q=c.q, raw=spoilt, table=(c.table, c.total))
        out, lse = d.attend(ctx)
        assert ctx.sync() == kvo.KVO_OK
        before = at - (n - tokens) if kind < 3 else tokens    # tokens that do not see it
        assert torch.equal(out[:before], clean[0][:before]) and torch.equal(lse[:before], clean[1][:before])
        assert torch.isnan(lse[before:]).all() and torch.isnan(out[before:, :, :64]).all()
    q = c.q.clone()                                           # a NaN query is its own columns' alone
    q[5, 3] = float("nan")
    d = Long(kvo, rng, [tokens], [n], heads, rows=400, q=q, raw=c.raw, table=(c.table, c.total))
    out, lse = d.attend(ctx)
    assert torch.isnan(out[5, 3]).all() and torch.isnan(lse[5, 3])
    out[5, 3], lse[5, 3] = clean[0][5, 3], clean[1][5, 3]
    # A column whose logits have no maximum sends its 256 columns through another pass, with other references r': their
    # weights 2^(z - r') are rounded to bf16 afresh, each by 2^-8 at most as before, so that the bits may change and the
    # bound stays.
    c.check_attend(out, lse)
    assert torch.equal(out[16:], clean[0][16:]) and torch.equal(lse[16:], clean[1][16:])


def test_long_chunk_infinite_logits(kvo, ctx):
    rng = np.random.default_rng(105)
    n, heads, tokens = 700, 20, 60
    raw = random_rows(rng, n)
    raw[3::7, 528:530] = np.array([0x7F80], np.uint16).view(np.uint8)             # +inf
    raw[:300, 528:530] = np.array([0x7F80], np.uint16).view(np.uint8)             # whole tiles of them
    q = np.abs(rng.standard_normal((tokens, heads, 576)))
    q[:, :, 512] = -np.abs(q[:, :, 512])
    c = Long(kvo, rng, [tokens], [n], heads, 0, q=dev(q, torch.bfloat16), raw=raw)
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    keys = C.values(raw)
    for t in range(tokens):
        seen = C.seen(c.starts, c.lens, 0, t, n)
        have = [p for p in range(300, seen) if p % 7 != 3]
        want, want_lse, spread, size = C.attend(f64(c.q)[t], SCALE, keys[have])
        tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 4 * U * 576 * size + 100 * U)[:, None]
        assert (np.abs(f64(out)[t] - want) <= tol).all()
        assert (np.abs(f64(lse)[t] - want_lse) <= 2 * U * 576 * size + 100 * U + 2 * U * np.abs(want_lse)).all()
    raw[:, 528:530] = np.array([0x7F80], np.uint16).view(np.uint8)
    c = Long(kvo, rng, [tokens], [n], heads, 0, q=c.q, raw=raw)
    out, lse = c.attend(ctx)
    assert ctx.sync() == kvo.KVO_OK
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("heads,tokens", [(64, 50), (128, 70)])
def test_long_chunk_bad_pages(kvo, ctx, heads, tokens):
    rng = np.random.default_rng([106, heads])
    table = np.array([[-1, 1, -5, 3, 0, 77, 2 ** 31 - 1], [2, 0, 77, 9999, -1, -1, -1]], np.int32)
    for lens, want in (([112, 60], kvo.KVO_ERANGE), ([80, 20], kvo.KVO_ERANGE), ([0, 32], kvo.KVO_OK)):
        c = Long(kvo, rng, [tokens, min(tokens, 7)], lens, heads, 16, rows=112, table=(table, 4))
        out, lse = c.attend(ctx)
        assert ctx.sync() == want
        c.check_attend(out, lse)


def test_long_chunk_bad_starts(kvo, ctx):
    rng = np.random.default_rng(107)
    c = Long(kvo, rng, [40, 40, 40], [100, 90, 80], 20)
    for starts in ([0, 40, 80, 121], [-1, 40, 80, 120], [0, 90, 40, 120], [0, 40, 2 ** 31 - 1, 120], [0, -2 ** 31, 80, 120]):
        wide = torch.full((122, 20, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        c.dev_starts = dev(starts, torch.int32)
        c.attend(ctx, out=wide[1:121], lse=torch.zeros(120, 20, device="cuda"))
        assert ctx.sync() == kvo.KVO_ERANGE, starts
        assert (wide[0] == 7).all() and (wide[121] == 7).all()


@pytest.mark.parametrize("counts,lens,heads", [([70], [300], 24), ([30, 41], [200, 99], 128), ([40, 41], [99, 200], 7)])
def test_long_chunk_strides(kvo, ctx, counts, lens, heads):
    rng = np.random.default_rng([108, heads])
    c = Long(kvo, rng, counts, lens, heads)
    want, want_lse = c.attend(ctx)
    c.check_attend(want, want_lse)
    wide = torch.full((c.tokens, 2 * heads, 592), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1::2, 8:584] = c.q
    across = torch.empty(heads, c.tokens, 576, dtype=torch.bfloat16, device="cuda")
    across.copy_(c.q.transpose(0, 1))
    for q in (wide[:, 1::2, 8:584], across.transpose(0, 1)):
        c.q = q
        out, lse = c.attend(ctx)
        assert ctx.sync() == kvo.KVO_OK
        c.check_attend(out, lse)
        assert ctx.sync() == kvo.KVO_OK


@pytest.mark.parametrize("counts,lens,heads", [([64] * 3, [5000, 777, 2000], 64), ([90, 300], [4000, 900], 64), ([600], [600], 16),
                                               ([1] * 40, [3000] * 40, 64), ([5] * 9, [3100] * 9, 20)])
def test_the_same_bits_every_time(kvo, ctx, counts, lens, heads):
    """One call behind the other, on the same inputs."""
    rng = np.random.default_rng([109, heads])
    for kind in (Long, Chunk):
        c = kind(kvo, rng, counts, lens, heads)
        out, lse = c.attend(ctx)
        weights = c.weights(ctx, lse)
        for _ in range(20):
            got = [c.attend(ctx) for _ in range(3)]
            sums = [c.weights(ctx, lse) for _ in range(6)]
            for o, l in got:
                assert torch.equal(o, out) and torch.equal(l, lse)
            for w in sums:
                assert torch.equal(w, weights)
        assert ctx.sync() == kvo.KVO_OK


@pytest.mark.parametrize("counts,lens,heads", [([20, 12], [300, 40], 20), ([64] * 3, [5000, 777, 2000], 64)])
def test_long_chunk_waits_that_run_out(kvo, counts, lens, heads):
    rng = np.random.default_rng([110, sum(counts)])
    c = kvo.Context(1, 64, 64)
    chunk = Long(kvo, rng, counts, lens, heads)
    want = [t.clone() for t in chunk.attend(c)]
    assert c.sync() == kvo.KVO_OK
    for clocks in WAITS:
        c.set_wait_clocks(clocks)
        got = chunk.attend(c)
        status = c.sync()
        assert status in ((kvo.KVO_ETIMEDOUT,) if clocks == 0 else (kvo.KVO_OK, kvo.KVO_ETIMEDOUT))
        assert c.sync() == kvo.KVO_OK
        c.set_wait_clocks()
        for again in (got if status == kvo.KVO_OK else None, chunk.attend(c)):
            for a, b in zip(again or (), want):
                assert torch.equal(a, b), clocks
        assert c.sync() == kvo.KVO_OK
    c.close()


def test_long_chunk_on_two_streams_and_replayed(kvo, ctx):
    """The same bits from two calls at once, and from two graphs at once on new inputs."""
    rng = np.random.default_rng(111)
    both = [Long(kvo, rng, [90, 40], [700, 300], 64), Long(kvo, rng, [33] * 5, [900, 33, 500, 64, 257], 20)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def run(c):
        out, lse = c.attend(ctx)
        return out, lse, c.weights(ctx, lse)

    want = [[t.clone() for t in run(c)] for c in both]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s in zip(both, streams):
            with torch.cuda.stream(s):
                got.append(run(c))
        torch.cuda.synchronize()
        for a, b in zip(want[0] + want[1], got[0] + got[1]):
            assert torch.equal(a, b)
    graphs = []
    for c in both:
        cache = c.cache
        out, lse = c.attend(ctx)                               # (the wide table is made outside the graph)
        blocks = -(-60_000 // c.br)
        table = torch.full((c.n, blocks), -1, dtype=torch.int32, device="cuda")
        table[:, :c.table.shape[1]] = dev(c.table)
        wide = kvo.Cache(rows=dev(c.raw), block_rows=c.br, table=table)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, l = ctx.attend_chunk(wide, c.q, c.dev_starts, c.dev_lens, c.scale, 60_000)
            w = ctx.attention_weights(cache, c.q, c.dev_starts, c.dev_lens, l, c.scale, c.rows)
        graphs.append((g, (o, l, w), wide))
    for c in both:
        c.q.copy_(c.q.roll(1, 0))
    want = [[t.clone() for t in run(c)] for c in both]
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, got, _), w in zip(graphs, want):
            for a, b in zip(got, w):
                assert torch.equal(a, b)
    assert ctx.sync() == kvo.KVO_OK


@pytest.mark.parametrize("scale", [-0.05, 0.0, 1.5])
@pytest.mark.parametrize("kind", [Chunk, Long])
def test_chunk_scales(kvo, ctx, kind, scale):
    rng = np.random.default_rng([112, int(scale * 100) + 10])
    c = kind(kvo, rng, [40, 12], [300, 150], 20, scale=scale, gain=0.2)
    out, lse = c.attend(ctx)
    weights = c.weights(ctx, lse)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    c.check_weights(weights, lse)


@pytest.mark.parametrize("heads", [16, 64])
def test_tokens_of_no_sequence(kvo, ctx, heads):
    """Every sequence empty, tokens all the same: nothing is written for them, and carried weights stay."""
    rng = np.random.default_rng([113, heads])
    for kind in (Chunk, Long):
        c = kind(kvo, rng, [0, 0, 0], [50, 0, 700], heads, after=40)
        out = torch.full((40, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((40, heads), 7.0, device="cuda")
        c.attend(ctx, out=out, lse=lse)
        assert (out == 7).all() and (lse == 7).all()
        carry = dev(rng.exponential(1.0, (3, 700)), torch.float32)
        got = c.weights(ctx, lse, carry=carry, keep=2.0)
        assert ctx.sync() == kvo.KVO_OK
        for s, n in enumerate(c.lens):
            assert torch.equal(got[s, :n], 2 * carry[s, :n]) and not got[s, n:].any()


def test_rows_far_into_a_cache(kvo, ctx):
    """Rows past 2^32 bytes, of both caches, and queries past 2^31 elements."""
    rng = np.random.default_rng(114)
    far = 6_600_000 // 16                                       # blocks; times 16 * 656 bytes
    kinds = [Chunk(kvo, rng, [5, 3], [200, 90], 20), Long(kvo, rng, [50], [700], 64)]
    store = torch.zeros((far + 200) * 16, 656, dtype=torch.uint8, device="cuda")
    for c in kinds:
        want = c.attend(ctx)
        sums = c.weights(ctx, want[1])
        store[far * 16:far * 16 + len(c.raw)] = dev(c.raw)
        table = np.full((c.n, 60_000 // 16), -1, np.int32)
        table[:, :c.table.shape[1]] = c.table + far
        cache = kvo.Cache(rows=store, block_rows=16, table=dev(table))
        rows = 60_000 if isinstance(c, Long) else c.rows
        wide = torch.empty_strided((c.tokens, c.heads, 576), (2 ** 31 // c.tokens // 8 * 8 + 64, 576, 1),
                                   dtype=torch.bfloat16, device="cuda")
        wide.copy_(c.q)
        for q in (c.q, wide):
            out, lse = ctx.attend_chunk(cache, q, c.dev_starts, c.dev_lens, c.scale, rows)
            got = ctx.attention_weights(cache, q, c.dev_starts, c.dev_lens, lse, c.scale, c.rows)
            if q is c.q:
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(got, sums)
            c.check_attend(out, lse)
            c.check_weights(got, lse)
        budget = 40
        to_table = dev(np.arange(c.n * 3, dtype=np.int32).reshape(c.n, 3) + far + 150)
        to = kvo.Cache(rows=store, block_rows=16, table=to_table)
        kept, lens, _ = ctx.shrink_cache(cache, to, sums, c.dev_lens, budget, first=1, last=2)
        assert ctx.sync() == kvo.KVO_OK
        for s in range(c.n):
            stay = C.keep(sums[s].cpu().numpy(), c.lens[s], budget, 1, 2)
            assert kept[s].tolist() == stay
            at = [O.row_of(c.table, c.total, 16, c.n, s, p) for p in stay]
            base = (far + 150 + 3 * s) * 16
            assert np.array_equal(store[base:base + budget].cpu().numpy(), c.raw[at])
        del wide
        torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["ties", "specials", "falling", "negative", "equal", "close"])
@pytest.mark.parametrize("budget", [1, 1_000, 225_000, 449_999])
def test_shrink_orders_of_many(kvo, ctx, kind, budget):
    """Hundreds of thousands of weights, more than stay in shared memory, over a few blocks named again and again."""
    rng = np.random.default_rng([115, len(kind), budget])
    n = 450_000
    w = {"ties": lambda: rng.integers(0, 5, n) * 0.25, "falling": lambda: -np.arange(n) * 0.5, "equal": lambda: np.full(n, 3.0),
         "negative": lambda: -rng.exponential(1.0, n), "close": lambda: 1.0 + rng.integers(0, 700, n) * 2.0 ** -23,
         "specials": lambda: rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42, 7.0, -7.0], n)}[kind]()
    w = dev(w[None], torch.float32)
    first, last = (0, 0) if budget < 100 else (3, 9)
    raw = random_rows(rng, 64 * 16)
    table = rng.integers(0, 64, (1, n // 16 + 1)).astype(np.int32)
    cache = kvo.Cache(rows=dev(raw), block_rows=16, table=dev(table))
    to = kvo.Cache(rows=torch.zeros(budget, 656, dtype=torch.uint8, device="cuda"), block_rows=budget)
    kept, lens, got = ctx.shrink_cache(cache, to, w, dev([n], torch.int32), budget, first=first, last=last)
    assert ctx.sync() == kvo.KVO_OK
    stay = C.keep(w[0].cpu().numpy(), n, budget, first, last)
    assert lens.tolist() == [budget] and kept[0].tolist() == stay
    assert torch.equal(got[0].view(torch.int32), w[0, stay].view(torch.int32))


@pytest.mark.parametrize("counts,lens,heads", [([1, 1, 1], [700, 33, 300], 40), ([1] * 5, [900] * 5, 64), ([2, 1], [400, 700], 30),
                                               ([1, 3], [600, 500], 33), ([9, 1, 1], [300, 2000, 40], 12), ([1, 1], [3000, 9], 128)])
def test_weights_of_few_columns_strided(kvo, ctx, counts, lens, heads):
    """Few columns a sequence, heads apart from each other, in tiles that cut a token's heads."""
    rng = np.random.default_rng([116, heads, len(counts)])
    c = Chunk(kvo, rng, counts, lens, heads)
    lse = c.lse()
    want = c.weights(ctx, lse)
    c.check_weights(want, lse)
    wide = torch.full((c.tokens, 2 * heads, 592), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1::2, 8:584] = c.q
    across = torch.empty(heads, c.tokens, 576, dtype=torch.bfloat16, device="cuda")
    across.copy_(c.q.transpose(0, 1))
    for q in (wide[:, 1::2, 8:584], across.transpose(0, 1)):
        c.q = q
        for window in (0, 1):
            got = c.weights(ctx, lse, window=window)
            assert ctx.sync() == kvo.KVO_OK
            c.check_weights(got, lse, window)


# ------------------------------------------------- decoding on in a shrunk cache
def row_is(row, kv, pos):
    """Whether a cache row is what the token kv [576] (64-bit values) at position pos becomes."""
    for g in range(8):
        q, bits = O.latent_group(kv[64 * g:64 * g + 64])
        assert int(row[512 + 2 * g:514 + 2 * g].view(np.uint16)[0]) == bits
        assert np.array_equal(row[64 * g:64 * g + 64].view(np.int8), q)
    exact = O.rotate(kv[512:], pos, FREQ, True)
    pair = np.repeat(np.abs(kv[512::2]) + np.abs(kv[513::2]), 2)
    # 2^-8 |x| for bf16; the sine, the cosine, two products and a sum in fp32, 8 u of the pair
    assert (np.abs(O.row_values(row)[1] - exact) <= 2.0 ** -8 * np.abs(exact) + 8 * U * pair).all()


@pytest.mark.parametrize("heads,steps,draft", [(20, 3, 1), (64, 2, 3)])
def test_decoding_on_in_a_shrunk_cache(kvo, ctx, heads, steps, draft):
    """Behind a cut a token's row is the next place and its rotation goes on from the old length; a second cut later on."""
    rng = np.random.default_rng([117, heads])
    budget, br, n = 60, 16, 200
    st = session(kvo, ctx, [118, heads], sizes=((120, 60), (60, 61)), heads=heads, budget=budget)
    outs = run_session(ctx, st)
    assert ctx.sync() == kvo.KVO_OK
    total, table = outs[7], st["table"]
    old = st["pieces"][-1]["lens"].clone()
    small_table, small_total = block_table(rng, 2, -(-(budget + steps * draft) // br))
    store = torch.full((small_total * br, 656), 0x5A, dtype=torch.uint8, device="cuda")
    small = kvo.Cache(rows=store, block_rows=br, table=dev(small_table))
    _, held, _ = ctx.shrink_cache(st["cache"], small, total, old, budget, 2, 8)
    seq = dev(np.repeat([0, 1], draft), torch.int32)
    step = dev(np.tile(np.arange(draft), 2), torch.int32)
    starts = dev(np.array([0, draft, 2 * draft]), torch.int32)
    for _ in range(steps):
        kv = dev(rng.standard_normal((2 * draft, 576)), torch.bfloat16)
        q = dev(rng.standard_normal((2 * draft, heads, 576)), torch.bfloat16)
        before = store.cpu().numpy()
        place, pos = held[seq.long()] + step, old[seq.long()] + step
        values = torch.empty(2 * draft, 576, dtype=torch.bfloat16, device="cuda")
        ctx.append_tokens(small, kv[:, :512], kv[:, 512:], pos, FREQ, seq=seq, place=place, out_bf16=values)
        held += draft
        old += draft
        out, lse = ctx.attend_chunk(small, q, starts, held, SCALE, budget + steps * draft)
        assert ctx.sync() == kvo.KVO_OK
        after = store.cpu().numpy()
        for i in range(2 * draft):
            at = O.row_of(small_table, small_total, br, 2, int(seq[i]), int(place[i]))
            row_is(after[at], f64(kv)[i], int(pos[i]))
            assert np.array_equal(np.concatenate(O.row_values(after[at])), f64(values)[i])
            before[at] = after[at]
        assert np.array_equal(before, after)                  # and nothing else was written
        c = Chunk(kvo, rng, [draft, draft], held.tolist(), heads, br, rows=budget + steps * draft, q=q, raw=after,
                  table=(small_table, small_total))
        c.check_attend(out, lse)
    # cut once more, into another cache: the rotation still goes on from the old length
    last = torch.zeros(2 * 48, 656, dtype=torch.uint8, device="cuda")
    again = kvo.Cache(rows=last, block_rows=48)
    mass = ctx.attention_weights(small, q, starts, held, lse, SCALE, budget + steps * draft)
    _, fewer, _ = ctx.shrink_cache(small, again, mass, held, 40, 2, 8)
    kv = dev(rng.standard_normal((2, 576)), torch.bfloat16)
    ctx.append_tokens(again, kv[:, :512], kv[:, 512:], old, FREQ, place=fewer)
    assert ctx.sync() == kvo.KVO_OK
    for s in range(2):
        row_is(last[48 * s + int(fewer[s])].cpu().numpy(), f64(kv)[s], int(old[s]))


def test_places_of_appended_tokens(kvo, ctx):
    """Places apart from positions, into keys too; replayed from a graph; the position itself gives the same bytes."""
    rng = np.random.default_rng(119)
    table = np.array([[3, 1, -1], [0, 4, 2]], np.int32)
    n = 6
    kv = dev(rng.standard_normal((n, 576)), torch.bfloat16)
    key = dev(rng.standard_normal((n, 128)), torch.bfloat16)
    rows = torch.zeros(5 * 16, 656, dtype=torch.uint8, device="cuda")
    keys = torch.zeros(5 * 16, 128, dtype=torch.bfloat16, device="cuda")
    cache = kvo.Cache(rows=rows, keys=keys, block_rows=16, table=dev(table))
    seq = dev([0, 1, 0, 1, -1, 1], torch.int32)
    pos = dev([5, 2 ** 31 - 1, 1_000_000, 0, 3, 77], torch.int32)
    place = dev([31, 47, 0, 20, 2 ** 31 - 1, 0], torch.int32)

    def run():
        ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], pos, FREQ, seq=seq, key=key, place=place)

    run()
    assert ctx.sync() == kvo.KVO_OK
    got, where = rows.cpu().numpy(), {}
    for i in (0, 1, 2, 3, 5):
        at = O.row_of(table, 5, 16, 2, int(seq[i]), int(place[i]))
        where[i] = at
        row_is(got[at], f64(kv)[i], int(pos[i]))
        assert torch.equal(keys[at], key[i])
    rest = [r for r in range(80) if r not in where.values()]
    assert not got[rest].any() and not keys[rest].any()
    want, want_keys = rows.clone(), keys.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    rows.zero_()
    keys.zero_()
    g.replay()
    assert ctx.sync() == kvo.KVO_OK and torch.equal(rows, want) and torch.equal(keys, want_keys)
    # a place that is the position gives what none gives
    rows.zero_()
    at = dev([3, 3], torch.int32)
    ctx.append_tokens(cache, kv[:2, :512], kv[:2, 512:], at, FREQ)
    plain = rows.clone()
    rows.zero_()
    ctx.append_tokens(cache, kv[:2, :512], kv[:2, 512:], at, FREQ, place=at)
    assert ctx.sync() == kvo.KVO_OK and torch.equal(rows, plain)


@pytest.mark.parametrize("pos,place", [(4, -1), (4, -2 ** 31), (-1, 4), (4, 33), (4, 48), (4, 2 ** 31 - 1)])
def test_places_without_a_row(kvo, ctx, pos, place):
    """A place past the table, in a page that is not there, or below zero, and a position below zero: said, not written."""
    kv = dev(np.random.default_rng(120).standard_normal((1, 576)), torch.bfloat16)
    rows = torch.full((4 * 16, 656), 0x5A, dtype=torch.uint8, device="cuda")
    cache = kvo.Cache(rows=rows, block_rows=16, table=dev(np.array([[2, 0, -1]], np.int32)))
    values = torch.full((1, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], dev([pos], torch.int32), FREQ, out_bf16=values,
                      place=dev([place], torch.int32))
    assert ctx.sync() == kvo.KVO_ERANGE
    assert (rows == 0x5A).all() and not values.any()
    for bad in (dev([place], torch.int64), dev([place, 0], torch.int32), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            ctx.append_tokens(cache, kv[:, :512], kv[:, 512:], dev([4], torch.int32), FREQ, place=bad)


# -------------------------------------------------- the kernel of many columns
class Many(Long):
    """Chunks that are sure to go through the kernel of many columns: its scratch holds their rows as bf16."""

    def attend(self, ctx, rows=60_000, **kw):
        need = self.kvo.kvo_attend_chunk_work_bytes(self.tokens, self.n, self.heads, rows)
        assert need >= self.n * rows * 1152
        return super().attend(ctx, rows, **kw)


@pytest.mark.parametrize("kind", [Chunk, Many])
@pytest.mark.parametrize("counts", [[90, 0, 40, 0], [0, 0, 64, 70, 0]])
def test_chunk_idle_sequences(kvo, ctx, kind, counts):
    """Sequences without tokens are not looked at: their pages may be gone, and they change nothing."""
    rng = np.random.default_rng([121, len(counts)])
    heads, lens = 64, [300, 700, 90, 513, 60][:len(counts)]
    c = kind(kvo, rng, counts, lens, heads)
    want = c.attend(ctx)
    weights = c.weights(ctx, want[1])
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(*want)
    table = c.table.copy()
    table[[s for s, n in enumerate(counts) if n == 0]] = -1
    d = kind(kvo, rng, counts, lens, heads, q=c.q, raw=c.raw, table=(table, c.total))
    out, lse = d.attend(ctx)
    got = d.weights(ctx, lse)
    assert ctx.sync() == kvo.KVO_OK
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(got, weights)


@pytest.mark.parametrize("table", [True, False])
@pytest.mark.parametrize("counts", [[4] * 20, [0] * 13 + [70] + [0] * 6, [70] + [0] * 18 + [33], [1, 40, 7, 0, 300] * 4])
def test_chunk_sequences_in_groups(kvo, ctx, counts, table):
    """More rows than the scratch takes at once: some sequences after the others, behind a table and without."""
    rng = np.random.default_rng([122, sum(counts)])
    rows, heads = 250_000, 128
    lens = [n + (37 * s) % 500 for s, n in enumerate(counts)]
    c = Chunk(kvo, rng, counts, lens, heads, 16, first=1, after=2)
    need = kvo.kvo_attend_chunk_work_bytes(c.tokens, c.n, heads, rows)
    assert 2 ** 31 < need < 2 ** 32 * 1.01 < c.n * rows * 1152
    if table:
        wide = np.full((c.n, rows // 16), -1, np.int32)
        wide[:, :c.table.shape[1]] = c.table
        cache = kvo.Cache(rows=dev(c.raw), block_rows=16, table=dev(wide))
    else:
        store = torch.zeros(c.n, rows, 656, dtype=torch.uint8, device="cuda")
        for s, n in enumerate(lens):
            at = [O.row_of(c.table, c.total, 16, c.n, s, p) for p in range(n)]
            store[s, :n] = dev(c.raw[at])
        cache = kvo.Cache(rows=store.view(-1, 656), block_rows=rows)
    out = torch.full((c.tokens, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.tokens, heads), 7.0, device="cuda")
    ctx.attend_chunk(cache, c.q, c.dev_starts, c.dev_lens, SCALE, rows, out=out, lse=lse)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    for x in (out, lse):
        assert (x[0] == 7).all() and (x[-2:] == 7).all()
    again = ctx.attend_chunk(cache, c.q, c.dev_starts, c.dev_lens, SCALE, rows)
    assert torch.equal(again[0][1:-2], out[1:-2]) and torch.equal(again[1][1:-2], lse[1:-2])
    torch.cuda.empty_cache()


def test_chunk_bad_starts_in_groups(kvo, ctx):
    rng = np.random.default_rng(123)
    c = Chunk(kvo, rng, [20] * 20, [100 + s for s in range(20)], 128)
    wide_table = np.full((20, 250_000 // 16), -1, np.int32)
    wide_table[:, :c.table.shape[1]] = c.table
    cache = kvo.Cache(rows=dev(c.raw), block_rows=16, table=dev(wide_table))
    good = c.starts
    for at, to in ((20, 401), (0, -1), (10, 390), (13, 2 ** 31 - 1), (7, -2 ** 31)):
        starts = good.copy()
        starts[at] = to
        wide = torch.full((402, 128, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((402, 128), 7.0, device="cuda")
        ctx.attend_chunk(cache, c.q, dev(starts, torch.int32), c.dev_lens, SCALE, 250_000, out=wide[1:401], lse=lse[1:401])
        assert ctx.sync() == kvo.KVO_ERANGE, starts
        for x in (wide, lse):
            assert (x[0] == 7).all() and (x[401] == 7).all()


@pytest.mark.parametrize("counts,heads,rows", [
    ([4], 64, 240_000), ([256], 1, 240_000), ([10, 10], 20, 60_000), ([17, 12, 9], 20, 60_000),   # one tile of columns after the other
    ([5, 4, 3, 6], 64, 60_000), ([4, 0, 8, 4, 1], 64, 60_000),              # two side by side, of one sequence and of two
    ([40], 128, 60_000), ([9, 31, 0, 17, 2], 64, 60_000),                   # four
    ([1, 70, 1, 1, 1], 128, 60_000), ([1] * 9 + [200] + [1] * 9, 64, 60_000),
    ([(3 * s) % 11 for s in range(300)], 64, 12_000), ([130] + [1] * 290, 100, 12_000)])
def test_chunk_tiles_side_by_side(kvo, ctx, counts, heads, rows):
    """Sequences of very unequal lengths and numbers of tokens, more of them than are listed at a time."""
    rng = np.random.default_rng([124, sum(counts), heads])
    lens = [(1 + 97 * s * s) % 900 if n < 2 else n + (61 * s) % 1100 for s, n in enumerate(counts)]
    if len(counts) > 20:
        lens = [n + (5 * s) % 40 for s, n in enumerate(counts)]
    c = Many(kvo, rng, counts, lens, heads, first=1, after=1)
    out = torch.full((c.tokens, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.tokens, heads), 7.0, device="cuda")
    c.attend(ctx, rows, out=out, lse=lse)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    for x in (out, lse):
        assert (x[0] == 7).all() and (x[-1] == 7).all()


@pytest.mark.parametrize("order", ["rising", "falling", "one", "steps"])
@pytest.mark.parametrize("tokens,heads", [(10, 20), (14, 20), (5, 64), (90, 64)])
def test_many_columns_wide_logits(kvo, ctx, order, tokens, heads):
    """Logits far above the first tile's: tiles done again, alone and beside others that are not."""
    rng = np.random.default_rng([125, tokens, len(order)])
    n = 1300
    raw = random_rows(rng, n)
    for j in range(n):
        x = np.zeros(64)
        x[:8] = {"rising": j / 20, "falling": (n - j) / 20, "one": 60.0 * (j == n * 3 // 5), "steps": 9.0 * (j // 129)}[order]
        raw[j, 528:] = np.ascontiguousarray(O.bf16_bits(x)).view(np.uint8)
    q = rng.standard_normal((tokens, heads, 576))
    q[..., 512:520] = np.linspace(-1, 4, heads)[None, :, None]
    c = Many(kvo, rng, [tokens], [n], heads, 0, scale=0.5, q=dev(q, torch.bfloat16), raw=raw)
    out, lse = c.attend(ctx, rows=240_000)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)


@pytest.mark.parametrize("counts,lens,heads", [([10], [1000], 20), ([13, 12], [1000, 300], 20), ([5] * 9, [3100 - 300 * s for s in range(9)], 64),
                                               ([200], [777], 3), ([40] * 5, [900] * 5, 64)])
def test_many_columns_same_bits(kvo, ctx, counts, lens, heads):
    """One call behind the other, and with waits that run out between them."""
    rng = np.random.default_rng([126, heads, len(counts)])
    c = Many(kvo, rng, counts, lens, heads)
    out, lse = c.attend(ctx, rows=240_000)
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    for _ in range(20):
        o, l = c.attend(ctx, rows=240_000)
        assert torch.equal(o, out) and torch.equal(l, lse)
    own = kvo.Context(1, 64, 64)
    for clocks in WAITS:
        own.set_wait_clocks(clocks)
        c.attend(own, rows=240_000)
        assert own.sync() in ((kvo.KVO_ETIMEDOUT,) if clocks == 0 else (kvo.KVO_OK, kvo.KVO_ETIMEDOUT))
        own.set_wait_clocks()
        o, l = c.attend(own, rows=240_000)
        assert own.sync() == kvo.KVO_OK and torch.equal(o, out) and torch.equal(l, lse)
    own.close()


@pytest.mark.parametrize("tokens,n", [(3, 300), (300, 300), (90, 5000)])
@pytest.mark.parametrize("heads", [16, 64])
def test_weights_past_the_largest_number(kvo, ctx, tokens, n, heads):
    """Log-sum-exps far below the logits: a weight beyond fp32 is infinite, however many tiles come after it; not NaN."""
    rng = np.random.default_rng([127, tokens, heads])
    raw = random_rows(rng, n, scale=(1e-4, 1e-3))
    c = Chunk(kvo, rng, [tokens], [n], heads, 0, raw=raw, scale=0.01)
    lse = c.lse()
    lse[: max(1, tokens // 3)] = -500.0                        # one after the other: all of it, and the first tiles' alone
    carry = dev(rng.exponential(1.0, (1, n)), torch.float32)
    got = c.weights(ctx, lse, carry=carry)
    assert ctx.sync() == kvo.KVO_OK
    assert torch.isinf(got[0, : n - tokens + 1]).all() and (got > 0).all()
    # token i sees the first n - tokens + 1 + i positions: those that only later tokens see get the later ones' weights
    few = c.weights(ctx, torch.where(lse == -500.0, -float("inf"), lse), carry=carry)
    behind = n - tokens + max(1, tokens // 3)
    assert torch.isinf(got[0, :behind]).all()
    assert torch.equal(got[0, behind:], few[0, behind:]) and torch.isfinite(few).all()


@pytest.mark.parametrize("counts,heads", [([1], 16), ([1, 1, 1], 64), ([40], 20), ([300], 128)])
@pytest.mark.parametrize("size", [0.0, 1000.0, -20480.0])
def test_weights_take_the_difference_first(kvo, ctx, counts, heads, size):
    """Logits and log-sum-exps that are large and nearly equal: a weight is as exact as their difference."""
    rng = np.random.default_rng([128, sum(counts), heads])
    lens = [max(n, 700) for n in counts]
    c = Chunk(kvo, rng, counts, lens, heads, 16, scale=1.0)
    # z = size * 1 + 1 * f with f in 32nds: every product and the sum are exact in fp32, and so is z - lse
    f = rng.integers(0, 32, len(c.raw)) / 32
    c.raw[:, 512:] = 0
    for j, v in enumerate(f):
        x = np.zeros(64)
        x[:2] = 1.0, v
        c.raw[j, 528:] = np.ascontiguousarray(O.bf16_bits(x)).view(np.uint8)
    c.cache = kvo.Cache(rows=dev(c.raw), block_rows=16, table=dev(c.table))
    q = torch.zeros(c.tokens, heads, 576)
    q[..., 512], q[..., 513] = size, 1.0
    c.q = dev(q, torch.bfloat16)
    assert (c.q[..., 512] == size).all()
    off = rng.integers(0, 64, (c.tokens, heads)) / 8
    lse = dev(size + off, torch.float32)
    assert np.array_equal(f64(lse), size + off)
    got = f64(c.weights(ctx, lse))
    assert ctx.sync() == kvo.KVO_OK
    for s in range(c.n):
        at = [O.row_of(c.table, c.total, 16, c.n, s, p) for p in range(lens[s])]
        want = np.zeros(c.rows)
        for t in C.tokens_of(c.starts, s):
            n = C.seen(c.starts, c.lens, s, t, c.rows)
            want[:n] += np.exp(f[at[:n]][:, None] - off[t][None, :]).sum(1)
        # |z - lse| <= 8: its product with log2 e (rounded, by a rounded constant) is off by 2 u of 11.6, 17 u of the
        # weight; the exponential 16 u, the sums 64 u
        tol = (17 + 16 + 64) * U * want
        assert (np.abs(got[s] - want) <= tol).all(), float((np.abs(got[s] - want) / np.maximum(tol, 1e-300)).max())


# ------------------------------------------------------------- the largest calls
@pytest.mark.parametrize("sequences", [4_096, 65_535])
def test_as_many_sequences_as_there_may_be(kvo, ctx, sequences):
    """One token of two heads in each of them, their weights, and a cut to two positions, against 64 bits as a whole."""
    g = torch.Generator(device="cuda")
    g.manual_seed(sequences)
    n, heads, br = sequences, 2, 8
    lens = torch.randint(0, br + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    raw = torch.randint(0, 256, (n * br, 656), generator=g, device="cuda", dtype=torch.uint8)
    raw.view(torch.int8)[:, :512].clamp_(-127, 127)
    raw.view(torch.float16)[:, 256:264] = (torch.rand(n * br, 8, generator=g, device="cuda") * 9e-3 + 1e-3).half()
    raw.view(torch.bfloat16)[:, 264:] = torch.randn(n * br, 64, generator=g, device="cuda").bfloat16()
    table = torch.randperm(n, generator=g, device="cuda")[:, None].int()
    q = torch.randn(n, heads, 576, generator=g, device="cuda").bfloat16()
    cache = kvo.Cache(rows=raw, block_rows=br, table=table)
    starts = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out, lse = ctx.attend_chunk(cache, q, starts, lens, SCALE, br)
    mass = ctx.attention_weights(cache, q, starts, lens, lse, SCALE, br)
    to_rows = torch.zeros(n * 2, 656, dtype=torch.uint8, device="cuda")
    kept, left, w = ctx.shrink_cache(cache, kvo.Cache(rows=to_rows, block_rows=2), mass, lens, 2, 1, 0)
    assert ctx.sync() == kvo.KVO_OK
    rows = raw.view(n, br, 656)[table[:, 0].long()]
    lat = (rows.view(torch.int8)[..., :512].float().unflatten(-1, (8, 64)) *
           rows.view(torch.float16)[..., 256:264].float()[..., None]).flatten(-2).bfloat16().double()
    keys = torch.cat([lat, rows.view(torch.bfloat16)[..., 264:].double()], -1)
    hidden = torch.arange(br, device="cuda") >= lens[:, None]
    z = torch.einsum("nhd,nrd->nhr", q.double(), keys) * SCALE
    size = float(torch.einsum("nhd,nrd->nhr", q.double().abs(), keys.abs()).max()) * SCALE
    z = z.masked_fill(hidden[:, None], -float("inf"))
    want_lse = torch.logsumexp(z, 2)
    live = lens > 0
    p = torch.where(live[:, None, None], torch.exp(z - want_lse[..., None]), 0.0)
    want, spread = torch.einsum("nhr,nrd->nhd", p, lat), torch.einsum("nhr,nrd->nhd", p, lat.abs())
    logit = 2 * U * 576 * size                                  # as at the top of this file
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + spread * (2.0 ** -8 + 2 * logit + 100 * U) + 2.0 ** -80).all()
    assert torch.isneginf(lse[~live]).all()
    assert ((lse.double() - want_lse)[live].abs() <= logit + 100 * U + 2 * U * want_lse[live].abs()).all()
    assert ((mass.double() - p.sum(1)).abs() <= p.sum(1) * (2 * logit + 100 * U + 8 * U * (size + 3)) + 2.0 ** -120).all()
    assert torch.equal(left, lens.clamp(max=2))
    order = mass.clone()
    order[:, 0] = float("inf")
    order[hidden] = -float("inf")
    pick = order.sort(dim=1, descending=True, stable=True).indices[:, :2].sort(1).values.int()
    pick[torch.arange(2, device="cuda") >= left[:, None]] = -1
    assert torch.equal(kept, pick)
    there = (kept >= 0)
    assert torch.equal(w, torch.where(there, mass.gather(1, kept.clamp(min=0).long()), 0.0))
    moved = rows.gather(1, kept.clamp(min=0).long()[..., None].expand(-1, -1, 656))
    assert torch.equal(to_rows.view(n, 2, 656)[there], moved[there])


def test_chunk_groups_replayed_with_strided_queries(kvo, ctx):
    """Groups of sequences from a graph on new inputs, queries with heads before tokens, on another stream."""
    rng = np.random.default_rng(129)
    counts, rows, heads = [4, 0, 33, 5] * 5, 250_000, 128
    c = Chunk(kvo, rng, counts, [n + 50 for n in counts], heads, 16)
    wide = np.full((c.n, rows // 16), -1, np.int32)
    wide[:, :c.table.shape[1]] = c.table
    cache = kvo.Cache(rows=dev(c.raw), block_rows=16, table=dev(wide))
    across = torch.empty(heads, c.tokens, 576, dtype=torch.bfloat16, device="cuda")
    across.copy_(c.q.transpose(0, 1))
    c.q = across.transpose(0, 1)
    work = torch.empty(kvo.kvo_attend_chunk_work_bytes(c.tokens, c.n, heads, rows), dtype=torch.uint8, device="cuda")
    out = torch.empty(c.tokens, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(c.tokens, heads, device="cuda")

    def run():
        ctx.attend_chunk(cache, c.q, c.dev_starts, c.dev_lens, SCALE, rows, out=out, lse=lse, work=work)

    run()
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    across.copy_(across.roll(1, 1))
    out.zero_()
    work.fill_(255)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    assert ctx.sync() == kvo.KVO_OK
    c.check_attend(out, lse)
