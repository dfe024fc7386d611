"""Refusals of the calls on prompt chunks and shrunk caches, without a GPU: with a blank context a good call gets as far
as the launch (and fails there for want of a device), a bad one is refused."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
A = 1 << 20                                    # an aligned address that is never touched
NAN, INF = float("nan"), float("inf")


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


def chunk(K, **kw):
    base = dict(q=A, starts=A, lens=A, out=A, lse=A, work=A, work_bytes=1 << 50, q_ld=64 * 576, q_head_ld=576, tokens=20,
                rows=128, heads=64, scale=0.07)
    return fill(K.kvo_chunk_query(), **{**base, **kw})


def weight(K, **kw):
    base = dict(q=A, starts=A, lens=A, lse=A, carry=A, out=A, work=A, work_bytes=1 << 50, q_ld=64 * 576, q_head_ld=576,
                carry_ld=128, out_ld=128, tokens=20, rows=128, window=0, heads=64, scale=0.07, keep=1.0)
    return fill(K.kvo_weight_query(), **{**base, **kw})


def shrink(K, **kw):
    base = dict(weights=A, lens=A, kept=A, new_lens=A, to_weights=A, weights_ld=128, kept_ld=40, to_weights_ld=40, rows=128,
                budget=40, first=4, last=8)
    return fill(K.kvo_shrink(), **{**base, **kw})


BAD_CACHE = [dict(block_rows=0), dict(blocks=0), dict(blocks=2 ** 31), dict(sequences=0), dict(table=A + 2),
             dict(table_blocks=-1), dict(table_ld=7), dict(table=None, sequences=101), dict(sequences=65536),
             dict(blocks=2 ** 31 - 1, block_rows=2 ** 31 - 1), dict(rows=None), dict(rows=A + 8)]
BAD_QUERY = [dict(q=None), dict(q=A + 8), dict(q_ld=568), dict(q_ld=580), dict(q_ld=2 ** 38), dict(q_ld=-576),
             dict(q_head_ld=568), dict(q_head_ld=577), dict(q_head_ld=2 ** 38), dict(q_head_ld=0), dict(starts=None),
             dict(starts=A + 2), dict(lens=None), dict(lens=A + 1), dict(lse=A + 2), dict(heads=0), dict(heads=129),
             dict(tokens=-1), dict(tokens=65536), dict(rows=-1), dict(rows=2 ** 31 - 255), dict(scale=NAN), dict(scale=INF)]


def run(ctx, call, *structs):
    return call(*(None if s is None else ctypes.addressof(s) for s in (ctx, *structs)), None)


def test_chunk_refusals(kvo, ctx):
    K, call = kvo, kvo.lib().kvo_attend_chunk
    good = lambda c={}, s={}: run(ctx, call, cache(K, **c), chunk(K, **s))
    assert good() == K.KVO_ECUDA
    assert good(dict(keys=None, key_type=9)) == K.KVO_ECUDA        # keys are not looked at
    assert good({}, dict(lse=None)) == K.KVO_ECUDA and good({}, dict(rows=0)) == K.KVO_ECUDA
    assert good({}, dict(tokens=1, q_ld=8)) == K.KVO_ECUDA and good({}, dict(heads=1, q_head_ld=8)) == K.KVO_ECUDA
    for none in ((None, cache(K), chunk(K)), (ctx, None, chunk(K)), (ctx, cache(K), None)):
        assert run(none[0], call, *none[1:]) == K.KVO_EINVAL
    for c in BAD_CACHE:
        assert good(c) == K.KVO_EINVAL, c
    for s in BAD_QUERY + [dict(out=None), dict(out=A + 8), dict(work=A + 8)]:
        assert good({}, s) == K.KVO_EINVAL, s
        many = dict(rows=100_000, tokens=500)                      # the kernel of many columns
        assert good({}, {**many, **s}) == K.KVO_EINVAL, s
    assert good({}, dict(tokens=0, q=None, out=None, work=None, work_bytes=0)) == K.KVO_OK
    assert good({}, dict(tokens=0, starts=None)) == K.KVO_EINVAL


def test_weight_refusals(kvo, ctx):
    K, call = kvo, kvo.lib().kvo_attention_weights
    good = lambda c={}, s={}: run(ctx, call, cache(K, **c), weight(K, **s))
    assert good() == K.KVO_ECUDA
    assert good({}, dict(carry=None, carry_ld=0)) == K.KVO_ECUDA and good({}, dict(window=2 ** 40)) == K.KVO_ECUDA
    assert good(dict(sequences=1), dict(out_ld=0, carry_ld=0)) == K.KVO_ECUDA
    for none in ((None, cache(K), weight(K)), (ctx, None, weight(K)), (ctx, cache(K), None)):
        assert run(none[0], call, *none[1:]) == K.KVO_EINVAL
    for c in BAD_CACHE:
        assert good(c) == K.KVO_EINVAL, c
    for s in BAD_QUERY + [dict(lse=None), dict(out=None), dict(out=A + 2), dict(carry=A + 1), dict(work=A + 2), dict(work=None),
                          dict(work_bytes=100), dict(out_ld=127), dict(carry_ld=127), dict(window=-1), dict(keep=NAN),
                          dict(keep=-INF)]:
        assert good({}, s) == K.KVO_EINVAL, s
    assert good({}, dict(rows=0, out=None, work=None, work_bytes=0)) == K.KVO_OK
    # without tokens the carried weights still move
    assert good({}, dict(tokens=0, q=None, lse=None, work=None, work_bytes=0)) == K.KVO_ECUDA
    assert good({}, dict(tokens=0, out=None)) == K.KVO_EINVAL


def test_shrink_refusals(kvo, ctx):
    K, call = kvo, kvo.lib().kvo_shrink_cache
    to = dict(rows=2 * A)
    good = lambda c={}, t={}, s={}: run(ctx, call, cache(K, **c), cache(K, **{**to, **t}), shrink(K, **s))
    assert good() == K.KVO_ECUDA
    assert good({}, {}, dict(to_weights=None, to_weights_ld=0)) == K.KVO_ECUDA
    assert good(dict(keys=None), dict(keys=None)) == K.KVO_ECUDA and good(dict(key_type=K.BF16), dict(keys=None)) == K.KVO_ECUDA
    assert good({}, dict(rows=A, table=2 * A)) == K.KVO_ECUDA      # one pool, other blocks
    for c in BAD_CACHE:
        assert good(c) == K.KVO_EINVAL and good({}, c) == K.KVO_EINVAL, c
    for c, t in ((dict(keys=None), {}), (dict(key_type=K.BF16), {}), ({}, dict(key_type=K.BF16)), ({}, dict(keys=A + 8)),
                 (dict(key_scales=None), {}), ({}, dict(key_scales=A + 1)), ({}, dict(rows=A)), (dict(sequences=2), {}),
                 (dict(key_type=5), dict(key_type=5))):
        assert good(c, t) == K.KVO_EINVAL, (c, t)
    for s in (dict(weights=None), dict(weights=A + 2), dict(lens=None), dict(lens=A + 3), dict(kept=None), dict(kept=A + 2),
              dict(new_lens=None), dict(new_lens=A + 1), dict(to_weights=A + 2), dict(rows=0), dict(rows=2 ** 31 - 255),
              dict(budget=0), dict(budget=2 ** 31 - 255), dict(first=-1), dict(last=-1), dict(first=20, last=21),
              dict(first=2 ** 31 - 1, last=2 ** 31 - 1), dict(weights_ld=127), dict(kept_ld=39), dict(to_weights_ld=39)):
        assert good({}, {}, s) == K.KVO_EINVAL, s
    for none in ((None, cache(K), cache(K, **to), shrink(K)), (ctx, None, cache(K, **to), shrink(K)),
                 (ctx, cache(K), None, shrink(K)), (ctx, cache(K), cache(K, **to), None)):
        assert run(none[0], call, *none[1:]) == K.KVO_EINVAL


def test_work_bytes(kvo, ctx):
    K = kvo
    for bad in ((-1, 1, 64, 10), (65536, 1, 64, 10), (1, 0, 64, 10), (1, 65536, 64, 10), (1, 1, 0, 10), (1, 1, 129, 10),
                (1, 1, 64, -1), (1, 1, 64, 2 ** 31 - 255)):
        assert K.kvo_attend_chunk_work_bytes(*bad) == -1, bad
        assert K.kvo_attention_weights_work_bytes(*bad) == -1, bad
    assert K.kvo_attention_weights_work_bytes(1, 1, 64, 10, -1) == -1
    assert K.kvo_attend_chunk_work_bytes(0, 1, 64, 10) == 0 and K.kvo_attention_weights_work_bytes(0, 1, 64, 10) == 0
    for tokens in (1, 7, 300, 65535):
        for sequences in (1, 5, 65535):
            for heads in (1, 20, 64, 128):
                for rows in (0, 1, 127, 5000, 2 ** 20, 2 ** 31 - 256):
                    need = K.kvo_attend_chunk_work_bytes(tokens, sequences, heads, rows)
                    assert need >= 0 and need % 4 == 0
                    assert 0 <= K.kvo_attention_weights_work_bytes(tokens, sequences, heads, rows) < 2 ** 24
    for tokens, rows in ((20, 2 ** 20), (500, 100_000)):           # parts to join; and values at hand for many columns
        need = K.kvo_attend_chunk_work_bytes(tokens, 3, 64, rows)
        for got, want in ((need, K.KVO_ECUDA), (need - 1, K.KVO_EINVAL)):
            if got >= 0:
                s = chunk(K, tokens=tokens, rows=rows, work_bytes=got)
                assert run(ctx, K.lib().kvo_attend_chunk, cache(K), s) == want
        if need:
            s = chunk(K, tokens=tokens, rows=rows, work=None)
            assert run(ctx, K.lib().kvo_attend_chunk, cache(K), s) == K.KVO_EINVAL


def test_work_bytes_are_bounded(kvo):
    """However many sequences there are and however long the longest may be."""
    K = kvo
    for tokens in (4, 64, 1_024, 4_096, 65_535):
        for sequences in (1, 3, 64, 256, 512, 65_535):
            for heads in (1, 16, 128):
                for rows in (1, 1_000, 131_072, 3_728_270, 10_000_000, 2 ** 31 - 256):
                    need = K.kvo_attend_chunk_work_bytes(tokens, sequences, heads, rows)
                    # 4 GiB of values, a factor a row, 76 pairs' parts of 128 columns, the plan
                    assert 0 <= need <= 2 ** 32 * (1 + 4 / 1152) + 2 ** 26, (tokens, sequences, heads, rows, need)
    # and no smaller than the rows need where these fit
    assert K.kvo_attend_chunk_work_bytes(1_024, 64, 16, 16_384) >= 64 * 16_384 * 1152


def test_binding_refuses_wrong_tensors(kvo):
    K = kvo
    c = ctypes.create_string_buffer(8192)
    paged = type("Paged", (), dict(sequences=2, ref=0))()
    starts, lens = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, lse = torch.zeros(4, 8, 576, dtype=torch.bfloat16), torch.zeros(4, 8)
    for bad in (q, q[0], q[..., :512], q.float()):                 # on the CPU, of two dimensions, short, of another type
        with pytest.raises((ValueError, TypeError)):
            K.kvo_attend_chunk(ctypes.addressof(c), paged, bad, starts, lens, 0.1, 64)
        with pytest.raises((ValueError, TypeError)):
            K.kvo_attention_weights(ctypes.addressof(c), paged, bad, starts, lens, lse, 0.1, 64)
    for bad in (torch.zeros(2, 64), torch.zeros(64), torch.zeros(2, 64, dtype=torch.float16)):
        with pytest.raises((ValueError, TypeError)):
            K.kvo_shrink_cache(ctypes.addressof(c), paged, paged, bad, lens, 10)


def test_binding_refuses_scratch_of_another_gpu(kvo):
    """Scratch has to be on the GPU of the queries; no second GPU is needed to see that."""
    class Scratch:
        dtype, is_cuda = torch.uint8, True

        def __init__(self, index):
            self.device = torch.device("cuda", index)

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return A

        def numel(self):
            return 512

    here = torch.device("cuda", 0)
    assert kvo._work(Scratch(0), 512, here, None)[1:] == (A, 512)
    assert kvo._work(None, 0, here, None) == (None, None, 0)
    with pytest.raises(ValueError, match="cuda:0"):
        kvo._work(Scratch(1), 512, here, None)


def test_no_copy_is_multicast():
    """Copies go to one CTA each: what they read may be memory that the caller names, of any kind."""
    import glob
    import os
    import re
    root = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gather_radix_top_gb300", "csrc")
    sources = glob.glob(os.path.join(root, "*.cu*"))
    assert len(sources) > 10
    for path in sources:
        text = open(path).read()
        assert "load_box_multicast" not in text, path
        for copy in re.findall(r"cp\.async\.bulk[^;]*;", text):
            assert "multicast" not in copy, (path, copy)
