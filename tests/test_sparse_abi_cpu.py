"""Refusals of the sparse decode calls, without a GPU.

Argument checks come before the context is looked at and before anything is
launched: with a blank context, a good call gets as far as the launch (and
fails there for want of a device), a bad one is refused."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20                                    # an aligned address that is never touched


@pytest.fixture(scope="module")
def kvo():
    from gather_radix_top_gb300 import build, kvo as K
    build.build()
    if torch.cuda.is_available():
        pytest.skip("would launch on the blank context's addresses")
    return K


@pytest.fixture()
def ctx():
    return ctypes.create_string_buffer(8192)


def fill(struct, **kw):
    for k, v in kw.items():
        setattr(struct, k, v)
    return struct


def cache(K, **kw):
    base = dict(rows=A, keys=A, key_scales=A, table=A, table_ld=8, blocks=100, block_rows=16, table_blocks=8,
                sequences=3, key_type=K.E4M3)
    return fill(K.kvo_cache(), **{**base, **kw})


FREQ = (ctypes.c_double * 32)(*[1.0] * 32)


def tokens(K, **kw):
    base = dict(latent=A, rope=A, key=A, seq=A, pos=A, inv_freq=ctypes.addressof(FREQ), out_bf16=A, latent_ld=576,
                rope_ld=576, key_ld=128, n=5, dtype=K.BF16, interleaved=1)
    return fill(K.kvo_tokens(), **{**base, **kw})


def score(K, **kw):
    base = dict(q=A, weights=A, lens=A, scores=A, q_ld=64 * 128, q_head_ld=128, weights_ld=64, ld=128, n=128,
                per_seq=2, heads=64, block=1)
    return fill(K.kvo_score_query(), **{**base, **kw})


def query(K, **kw):
    base = dict(q=A, lens=A, sel=A, out=A, lse=A, work=A, work_bytes=1 << 40, q_ld=64 * 576, q_head_ld=576,
                sel_ld=128, rows=0, picked=128, sel_block=1, per_seq=2, heads=64, scale=0.07)
    return fill(K.kvo_attend_query(), **{**base, **kw})


BAD_CACHE = [dict(block_rows=0), dict(blocks=0), dict(blocks=2 ** 31), dict(sequences=0), dict(table=A + 2),
             dict(table_blocks=-1), dict(table_ld=7), dict(table=None, sequences=101),
             dict(blocks=2 ** 31 - 1, block_rows=2 ** 31 - 1)]
BAD_ROWS = [dict(rows=None), dict(rows=A + 8)]
BAD_KEYS = [dict(keys=None), dict(keys=A + 8), dict(key_scales=None), dict(key_scales=A + 2), dict(key_type=1),
            dict(key_type=2), dict(key_type=7)]


def run(K, ctx, call, c, q):
    return call(ctypes.addressof(ctx) if ctx is not None else None, ctypes.addressof(c) if c is not None else None,
                ctypes.addressof(q) if q is not None else None, None)


def test_append_refusals(kvo, ctx):
    K, call = kvo, kvo.lib().kvo_append_tokens
    good = lambda c={}, t={}: run(K, ctx, call, cache(K, **c), tokens(K, **t))
    assert good() == K.KVO_ECUDA
    assert run(K, None, call, cache(K), tokens(K)) == K.KVO_EINVAL
    assert run(K, ctx, call, None, tokens(K)) == K.KVO_EINVAL
    assert run(K, ctx, call, cache(K), None) == K.KVO_EINVAL
    for c in BAD_CACHE + BAD_ROWS + BAD_KEYS:
        assert good(c) == K.KVO_EINVAL, c
    for c in (dict(keys=None), dict(key_type=7)):                  # keys are not looked at without a key
        assert good(c, dict(key=None)) == K.KVO_ECUDA, c
    nan, big = (ctypes.c_double * 32)(*[1.0] * 31, float("nan")), (ctypes.c_double * 32)(2.0 ** 21)
    for t in (dict(n=-1), dict(latent=None), dict(rope=None), dict(pos=None), dict(latent=A + 8), dict(rope=A + 2),
              dict(key=A + 4), dict(seq=A + 2), dict(pos=A + 1), dict(out_bf16=A + 8), dict(latent_ld=580),
              dict(latent_ld=504), dict(rope_ld=56), dict(key_ld=120), dict(dtype=K.E4M3), dict(dtype=-1),
              dict(inv_freq=None), dict(inv_freq=ctypes.addressof(nan)), dict(inv_freq=ctypes.addressof(big))):
        assert good({}, t) == K.KVO_EINVAL, t
    assert good({}, dict(dtype=K.FP32, latent_ld=516)) == K.KVO_ECUDA     # 16 bytes either way
    assert good({}, dict(n=0, latent=None, rope=None, pos=None)) == K.KVO_OK
    assert good(dict(table=None), dict(seq=None)) == K.KVO_ECUDA


def test_score_refusals(kvo, ctx):
    K, call = kvo, kvo.lib().kvo_index_scores
    good = lambda c={}, s={}: run(K, ctx, call, cache(K, **c), score(K, **s))
    assert good() == K.KVO_ECUDA
    assert good(dict(rows=None)) == K.KVO_ECUDA
    assert good(dict(key_type=K.BF16, key_scales=None)) == K.KVO_ECUDA
    for c in BAD_CACHE + BAD_KEYS:
        assert good(c) == K.KVO_EINVAL, c
    for s in (dict(q=None), dict(weights=None), dict(lens=None), dict(scores=None), dict(q=A + 8), dict(q_ld=8200),
              dict(q_head_ld=136), dict(weights=A + 2), dict(lens=A + 1), dict(scores=A + 2), dict(heads=0),
              dict(heads=129), dict(per_seq=0), dict(n=0), dict(n=-5), dict(n=2 ** 31 - 255, ld=2 ** 31), dict(ld=127),
              dict(block=0), dict(block=3), dict(block=256), dict(block=-2), dict(per_seq=30000)):
        assert good({}, s) == K.KVO_EINVAL, s
    assert good({}, dict(block=16, ld=8)) == K.KVO_ECUDA
    assert good({}, dict(block=16, ld=7)) == K.KVO_EINVAL


def test_attend_refusals(kvo, ctx):
    K, call = kvo, kvo.lib().kvo_attend
    good = lambda c={}, q={}: run(K, ctx, call, cache(K, **c), query(K, **q))
    assert good() == K.KVO_ECUDA
    assert good(dict(keys=None, key_type=9)) == K.KVO_ECUDA
    assert good({}, dict(sel=None, rows=128, lse=None)) == K.KVO_ECUDA
    assert good({}, dict(picked=0)) == K.KVO_ECUDA and good({}, dict(sel=None, rows=0)) == K.KVO_ECUDA
    for c in BAD_CACHE + BAD_ROWS:
        assert good(c) == K.KVO_EINVAL, c
    for q in (dict(q=None), dict(lens=None), dict(out=None), dict(q=A + 8), dict(q_ld=570), dict(q_head_ld=577),
              dict(lens=A + 2), dict(sel=A + 2), dict(out=A + 8), dict(lse=A + 2), dict(work=A + 8), dict(heads=0),
              dict(heads=129), dict(per_seq=0), dict(picked=-1), dict(sel_ld=127), dict(sel_block=0),
              dict(sel_block=24), dict(sel_block=256), dict(picked=2 ** 25, sel_ld=2 ** 25, sel_block=64),
              dict(sel=None, rows=-1), dict(sel=None, rows=2 ** 31 - 255), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(per_seq=30000)):
        assert good({}, q) == K.KVO_EINVAL, q


def test_attend_work_bytes(kvo):
    w = kvo.kvo_attend_work_bytes
    for bad in ((0, 64, 10), (65536, 64, 10), (1, 0, 10), (1, 129, 10), (1, 64, -1), (1, 64, 2 ** 31 - 255)):
        assert w(*bad) == -1, bad
    for nq in (1, 7, 300):
        for heads in (1, 20, 64, 128):
            for n in (0, 1, 127, 2048, 2 ** 20):
                assert 0 <= w(nq, heads, n) < 2 ** 31


def test_too_little_work_space(kvo, ctx):
    K = kvo
    need = K.kvo_attend_work_bytes(6, 64, 2 ** 20)
    for got, want in ((need, K.KVO_ECUDA), (need - 1, K.KVO_EINVAL)):
        if got < 0:
            continue
        q = query(K, sel=None, rows=2 ** 20, work_bytes=got)
        assert run(K, ctx, K.lib().kvo_attend, cache(K), q) == want
    if need:
        assert run(K, ctx, K.lib().kvo_attend, cache(K), query(K, sel=None, rows=2 ** 20, work=None)) == K.KVO_EINVAL


def test_pool_rows_refusals(kvo):
    p, b, r = ctypes.c_void_p(), ctypes.c_int64(), ctypes.c_int32()
    assert kvo.lib().kvo_pool_rows(None, ctypes.byref(p), ctypes.byref(b), ctypes.byref(r)) == kvo.KVO_EINVAL


def test_binding_refuses_wrong_tensors(kvo):
    K = kvo
    cpu = torch.zeros(16, 656, dtype=torch.uint8)
    with pytest.raises(ValueError):
        K.Cache(rows=cpu, block_rows=16)
    with pytest.raises(ValueError):
        K.Cache(block_rows=16)
    with pytest.raises(ValueError):
        K.Cache(rows=cpu, block_rows=0)
    with pytest.raises(ValueError):
        K.Cache(keys=torch.zeros(16, 128), block_rows=16)


def test_bad_pages_have_no_row(tmp_path):
    """The device's own row lookup, compiled for the host and run on tables with bad entries."""
    from gather_radix_top_gb300 import build
    from oracle import kvo_sparse_oracle as O
    src = tmp_path / "rows.cu"
    src.write_text("""
#include <cstdio>
#include "kvo_cache.cuh"
int main() {
  int32_t table[2][4] = {{3, -1, 0, 2147483647}, {99, 7, 100, 5}};
  kvo::CacheView c = {nullptr, nullptr, nullptr, &table[0][0], 4, 100, 16, 3, 2, kvo::divider(16)};
  for (uint32_t s = 0; s < 2; ++s)
    for (uint32_t p = 0; p < 80; ++p) std::printf("%lld\\n", (long long)kvo::cache_row(c, s, p));
  std::printf("%lld\\n", (long long)kvo::cache_row(c, 1, 2147483647u));
  kvo::CacheView d = {nullptr, nullptr, nullptr, nullptr, 0, 4000000, 1000, 0, 4000000,
                      kvo::divider(1000)};
  uint64_t wrong = 0;
  const uint32_t around[] = {1, 2, 3, 5, 7, 16, 48, 1000, 12345, 65535, 65536, 99999, 2147483647u};
  for (uint32_t x : around) {
    const kvo::Divider by = kvo::divider(x);
    for (uint64_t k = 0; k < 200000; ++k) {
      const uint64_t base = k * 10737ull / x * x;
      for (int64_t e = -1; e <= 1; ++e) {
        const int64_t n = (int64_t)base + e;
        if (n >= 0 && n < 2147483648ll) wrong += kvo::divide((uint32_t)n, by) != (uint32_t)n / x;
      }
    }
    wrong += kvo::divide(2147483647u, by) != 2147483647u / x;
  }
  std::printf("%llu\\n", (unsigned long long)wrong);
  std::printf("%lld %lld\\n", (long long)kvo::cache_row(d, 3999999, 999), (long long)kvo::cache_row(d, 5, 1000));
}
""")
    exe = tmp_path / "rows"
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", str(exe),
                    str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    table = np.array([[3, -1, 0], [99, 7, 100]])
    want = [O.row_of(table, 100, 16, 2, s, p) for s in range(2) for p in range(80)]
    assert got[:160] == [-1 if w is None else w for w in want]
    assert got[160:] == [-1, 0, 3999999999, -1]


def test_wait_clocks_refusals(kvo, ctx):
    call = kvo.lib().kvo_debug_set_wait_clocks
    assert call(None, 5) == kvo.KVO_EINVAL
    assert call(ctypes.addressof(ctx), -1) == kvo.KVO_EINVAL
    assert call(ctypes.addressof(ctx), 0) == kvo.KVO_OK


def test_turns_of_either_sign(tmp_path):
    """inv_freq / 2 pi modulo one turn, in units of 2^-64: off by at most one unit for each of the two parts it is put
    together from, whatever the sign (an angle at position 2^31 - 1 is off by 2^-32 turns at most)."""
    from fractions import Fraction
    from gather_radix_top_gb300 import build
    src = tmp_path / "turns.cu"
    src.write_text("""
#include <cstdio>
#include <cstdlib>
#include "kvo_append.cu"
kvo_status kvo::usable_status(kvo_ctx*, uint32_t**, int64_t*) { return KVO_ECUDA; }
int kvo::device_sms() { return 1; }
int main(int argc, char** argv) {
  for (int i = 1; i < argc; ++i)
    std::printf("%llu\\n", (unsigned long long)kvo::turns_of(std::strtod(argv[i], nullptr)));
}
""")
    exe = tmp_path / "turns"
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", str(exe),
                    str(src)], check=True)
    rng = np.random.default_rng(3)
    x = [0.0, 1.0, 1e-5, 3e-9, 1e-15, 2.0 ** -40, 0.7, 6.283185307179586, 1234.5, 2.0 ** 20, 1e-30, 5e-324]
    x += list(np.exp(rng.uniform(np.log(1e-20), np.log(2.0 ** 20), 200)))
    x = [s * v for v in x for s in (1.0, -1.0)]
    got = subprocess.run([str(exe), *[float(v).hex() for v in x]], check=True, capture_output=True, text=True).stdout.split()
    two_pi = Fraction(62831853071795864769252867665590057683943387987502116419498891846156328125724179972560696506842341359,
                      10 ** 100)
    for v, g in zip(x, got):
        want = Fraction(v) / two_pi * 2 ** 64
        off = (Fraction(int(g)) - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 2, (v, float(min(off, 2 ** 64 - off)))
