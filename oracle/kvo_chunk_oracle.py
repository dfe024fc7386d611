"""Prompt chunks over cached rows, and caches shrunk by attention weight, in 64
bits and plain loops: what kvo_attend_chunk, kvo_attention_weights and
kvo_shrink_cache have to return."""
import numpy as np

from . import kvo_sparse_oracle as S


def values(rows) -> np.ndarray:
    """The 576 values that each 656-byte row stands for."""
    return np.stack([np.concatenate(S.row_values(r)) for r in rows]) if len(rows) else np.zeros((0, 576))


def tokens_of(starts, s) -> range:
    return range(int(starts[s]), int(starts[s + 1]))


def seen(starts, lens, s, t, rows) -> int:
    """The positions that token t of sequence s sees."""
    n, i = int(starts[s + 1]) - int(starts[s]), t - int(starts[s])
    return min(max(int(lens[s]) - n + 1 + i, 0), rows)


def attend(q, scale, keys):
    """q [H, 576] against keys [n, 576]: (out [H, 512], lse [H], spread [H, 512] = sum p |v|, size [H] = the largest
    scale * sum |q k|)."""
    heads, lat = q.shape[0], keys[:, :S.LATENT]
    if not len(keys):
        return np.zeros((heads, S.LATENT)), np.full(heads, -np.inf), np.zeros((heads, S.LATENT)), np.zeros(heads)
    z = scale * (q @ keys.T)
    top = z.max(1, keepdims=True)
    p = np.exp(z - top)
    total = p.sum(1, keepdims=True)
    p /= total
    return p @ lat, (np.log(total) + top)[:, 0], p @ np.abs(lat), abs(scale) * (np.abs(q) @ np.abs(keys).T).max(1)


def weights(q, scale, keys, lse):
    """What q [H, 576] with log-sum-exps lse [H] gives to keys [n, 576]: (sums [n], and each term's share of an error in
    its logit [n] = sum_h p * (scale * sum |q k| + |lse|))."""
    live = ~np.isneginf(lse)
    z = scale * (q[live] @ keys.T)
    p = np.exp(z - lse[live, None])
    size = abs(scale) * (np.abs(q[live]) @ np.abs(keys).T) + np.abs(lse[live, None])
    return p.sum(0), (p * size).sum(0)


def keep(weights, length, budget, first, last) -> list:
    """The positions that stay, one after the other taken: the protected ones, then the largest weight left, of equal ones
    the lowest position, NaN last."""
    if length <= budget:
        return list(range(length))
    taken = set(range(min(first, length))) | set(range(max(0, length - last), length))
    rank = [(np.isnan(w), -w if not np.isnan(w) else 0.0, p) for p, w in enumerate(weights[:length].tolist())]
    for _, _, p in sorted(rank):
        if len(taken) >= budget:
            break
        taken.add(p)
    return sorted(taken)
