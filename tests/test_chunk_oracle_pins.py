"""The 64-bit oracle of prompt chunks and shrunk caches against independent forms."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from oracle import kvo_chunk_oracle as C

STARTS, LENS = np.array([2, 5, 5, 9]), [7, 40, 2]


def test_a_token_sees_the_positions_up_to_its_own():
    """Token i of n stands at position lens - n + i; a causal mask over the whole sequence says the same."""
    for s, n in enumerate(LENS):
        tokens = list(C.tokens_of(STARTS, s))
        mask = np.tril(np.ones((n, n), bool))[max(n - len(tokens), 0):]
        mask = np.concatenate([np.zeros((len(tokens) - len(mask), n), bool), mask])
        for t, row in zip(tokens, mask):
            assert C.seen(STARTS, LENS, s, t, 1000) == row.sum()
            assert C.seen(STARTS, LENS, s, t, 3) == row[:3].sum()
    assert [C.seen(STARTS, LENS, 2, t, 1000) for t in range(5, 9)] == [0, 0, 1, 2]


def test_attend_and_weights_against_torch():
    rng = np.random.default_rng(1)
    q, keys, scale = rng.standard_normal((4, 576)), rng.standard_normal((31, 576)) * 0.2, 0.07
    out, lse, spread, size = C.attend(q, scale, keys)
    z = scale * torch.tensor(q) @ torch.tensor(keys).T
    p = torch.softmax(z, -1)
    assert np.allclose(out, p @ torch.tensor(keys[:, :512])) and np.allclose(lse, torch.logsumexp(z, -1))
    assert (spread >= np.abs(out)).all() and (size[:, None] >= z.abs().numpy()).all()
    w, share = C.weights(q, scale, keys, lse)
    assert np.allclose(w, p.sum(0)) and np.isclose(w.sum(), 4) and (share >= 0).all()
    lse[2] = -np.inf
    assert np.allclose(C.weights(q, scale, keys, lse)[0], p[[0, 1, 3]].sum(0))
    out, lse, _, _ = C.attend(q, scale, keys[:0])
    assert not out.any() and np.isneginf(lse).all()


def test_values_of_no_rows():
    assert C.values([]).shape == (0, 576)


@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (5, 2, 2), (9, 0, 9), (9, 9, 0), (20, 3, 4)])
def test_keep_against_a_stable_sort(budget, first, last):
    rng = np.random.default_rng(budget)
    w = rng.integers(0, 4, 20).astype(np.float32)
    w[[3, 11]] = np.nan, np.inf
    key = np.where(np.isnan(w), np.inf, -w)
    key[:first], key[len(w) - last:] = -np.inf, -np.inf            # (an infinite weight ties with these, but they fit all)
    got = C.keep(w, 20, budget, first, last)
    assert got == sorted(got) and len(got) == min(budget, 20)
    assert set(range(first)) | set(range(20 - last, 20)) <= set(got)
    rest = [p for p in np.argsort(key, kind="stable") if first <= p < 20 - last]
    assert set(got) - set(range(first)) - set(range(20 - last, 20)) == set(int(p) for p in rest[:budget - first - last])
    if budget >= 4:
        assert C.keep(w, 4, budget, first, last) == [0, 1, 2, 3]
