"""The 64-bit oracle of the sparse decode operators, against independent forms."""
import math

import numpy as np
import pytest

from oracle import kvo_sparse_oracle as O

torch = pytest.importorskip("torch")


def test_bf16_rounding_matches_torch():
    x = np.random.default_rng(0).standard_normal(4000).astype(np.float32).astype(np.float64)
    x = np.concatenate([x, x * 1e-38, x * 1e38, [0.0, -0.0, np.inf, -np.inf, 1.00390625, 1.01171875]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(O.bf16_bits(x), want)


def test_e4m3_rounding_matches_torch():
    x = np.concatenate([np.random.default_rng(1).uniform(-448, 448, 2000), np.random.default_rng(2).normal(0, 0.01, 2000),
                        O._E4M3, (O._E4M3[:-1] + O._E4M3[1:]) / 2, [-0.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(np.array([O.e4m3_bits(float(v)) for v in x], np.uint8), want)
    vals = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.e4m3_value(np.arange(256)), vals.astype(np.float64), equal_nan=True)


def test_group_scale_is_the_smallest_that_holds_the_group():
    rng = np.random.default_rng(3)
    for k in range(200):
        x = rng.standard_normal(64).astype(np.float32) * np.float32(10.0) ** rng.integers(-9, 7)
        q, bits = O.latent_group(x)
        s = float(np.uint16(bits).view(np.float16))
        amax = float(np.abs(x.astype(np.float64)).max())
        assert 127 * s >= amax
        if bits > 0:
            assert 127 * float(np.uint16(bits - 1).view(np.float16)) < amax
            assert np.all(np.abs(q * s - x) <= s / 2)


def test_group_edges():
    q, bits = O.latent_group(np.zeros(64))
    assert bits == 0 and not q.any()
    x = np.zeros(64)
    x[3] = 2.0 ** -60
    q, bits = O.latent_group(x)                       # rounds up to the smallest fp16, which holds it as 0
    assert bits == 1 and not q.any()
    x[3] = 1e30
    q, bits = O.latent_group(x)
    assert bits == 0x7BFF and q[3] == 127
    x[3] = np.nan
    q, bits = O.latent_group(x)
    assert bits == 0x7E00 and not q.any()


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_matches_a_complex_product(interleaved):
    rng = np.random.default_rng(4)
    inv = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    x = rng.standard_normal(64)
    for pos in (0, 1, 777, 12345):
        got = O.rotate(x, pos, inv, interleaved)
        z = (x[0::2] + 1j * x[1::2]) if interleaved else (x[:32] + 1j * x[32:])
        z = z * np.exp(1j * pos * inv)
        want = np.empty(64)
        if interleaved:
            want[0::2], want[1::2] = z.real, z.imag
        else:
            want[:32], want[32:] = z.real, z.imag
        assert np.abs(got - want).max() < 1e-11
    # a rotation keeps lengths, however far the position
    far = O.rotate(x, 2 ** 31 - 1, inv, interleaved)
    assert abs(np.linalg.norm(far) - np.linalg.norm(x)) < 1e-12


def test_attend_against_torch():
    rng = np.random.default_rng(5)
    rows = rng.integers(0, 256, (37, 656), dtype=np.uint8)
    rows[:, 512:528] = rng.uniform(1e-3, 1e-2, (37, 8)).astype(np.float16).view(np.uint8)
    rows[:, 528:] = np.ascontiguousarray(O.bf16_bits(rng.standard_normal((37, 64)))).view(np.uint8)
    q = rng.standard_normal((5, 576))
    out, lse, spread, _ = O.attend(q, 0.07, list(rows))
    r = torch.from_numpy(rows)
    lat = (r[:, :512].view(torch.int8).float().view(37, 8, 64)
           * r[:, 512:528].contiguous().view(torch.float16).float()[:, :, None]).view(37, 512).bfloat16().double()
    key = torch.cat([lat, r[:, 528:].contiguous().view(torch.bfloat16).double()], 1)
    z = torch.from_numpy(q) @ key.T * 0.07
    assert np.allclose(out, (torch.softmax(z, 1) @ lat).numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(lse, torch.logsumexp(z, 1).numpy(), rtol=1e-13)
    assert (spread >= np.abs(out) - 1e-15).all()
    empty = O.attend(q, 0.07, [])
    assert not empty[0].any() and np.isneginf(empty[1]).all()


def test_positions_and_rows():
    assert O.positions_of(None, 1, 5, 3) == [0, 1, 2]
    assert O.positions_of([2, -1, 0], 4, 10, 0) == [8, 9, 0, 1, 2, 3]
    table = np.array([[3, -1], [0, 9]])
    assert O.row_of(table, 4, 16, 2, 0, 5) == 53
    assert O.row_of(table, 4, 16, 2, 0, 17) is None and O.row_of(table, 4, 16, 2, 1, 17) is None
    assert O.row_of(table, 4, 16, 2, 1, 32) is None
    assert O.row_of(None, 4, 16, 4, 2, 3) == 35 and O.row_of(None, 4, 16, 4, 2, 16) is None


def test_block_scores_are_maxima():
    rng = np.random.default_rng(6)
    q, w = rng.standard_normal((2, 3, 128)), rng.standard_normal((2, 3))
    keys = rng.standard_normal((20, 128))
    keys[4] = math.nan
    rows = [list(range(20)), list(range(19, -1, -1))]
    one, _ = O.index_scores(q, w, keys, np.ones(20), rows, [20, 7], 1)
    four, _ = O.index_scores(q, w, keys, np.ones(20), rows, [20, 7], 4)
    assert np.isnan(one[0, 4]) and np.isneginf(one[1, 7:]).all()
    want = np.where(np.isnan(one), -np.inf, one).reshape(2, 5, 4).max(2)
    assert np.array_equal(four, want)
