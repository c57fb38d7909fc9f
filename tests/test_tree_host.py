"""Trees of drafted tokens without a GPU: the oracle against closed forms, and the calls' refusals, which return before
any launch."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import tree as tr


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_29_gb300 import build
    build.build()
    import paged_kv_attention_29_gb300 as pkv
    return pkv.load()


def test_mask_words_round_trip():
    sees = np.random.default_rng(1).random((130, 130)) < 0.5
    assert np.array_equal(tr.sees_of(tr.words_of(sees, 3), 130), sees)


def test_a_chain_is_causal_attention():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(5, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    out, _ = tr.attention(q, k, v, np.tril(np.ones((5, 5), bool)), 0.3)
    for i in range(5):
        for h in range(4):
            s = k[:5 + i, h // 2] @ q[i, h] * 0.3
            p = np.exp(s) / np.exp(s).sum()
            assert np.allclose(out[i, h], p @ v[:5 + i, h // 2])


def test_rows_that_see_nothing_and_hidden_values():
    q, k, v = np.ones((2, 1, 4)), np.ones((2, 1, 4)), np.full((2, 1, 4), np.nan)
    v[1] = 3.0
    out, _ = tr.attention(q, k, v, np.array([[False, False], [False, True]]), 1.0)
    assert not out[0].any() and (out[1] == 3.0).all()


def test_accepted_paths():
    #      0
    #    1   2      (both hold the token sampled at 0: the first is taken)
    #    3   4
    sees = np.array([[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [1, 0, 1, 0, 1]], bool)
    assert tr.accept([7, 8, 9, 5, 6], [0, 7, 7, 8, 9], sees, 9) == ([0, 1, 3], 5)
    assert tr.accept([7, 1, 9, 5, 6], [0, 7, 7, 8, 9], sees, 9) == ([0, 1], 1)
    assert tr.accept([7, 8, 9, 5, 6], [0, 1, 7, 8, 9], sees, 9) == ([0, 2, 4], 6)
    assert tr.accept([7, 8, 9, 5, 6], [0, 1, 7, 8, 9], sees, 2) == ([0, 2], 9)
    assert tr.accept([3], [0], sees[:1, :1], 4) == ([0], 3)
    assert tr.accept([], [], sees[:0, :0], 4) == ([], -1)


P = None
X = ctypes.c_void_p(4096)        # non-null and aligned, never dereferenced: the checks return first


def attend(lib, fp8=False, words=1, batch=2, total=10, nodes=9, ctx=100, hq=16, hkv=8, d=128, bs=256, nb=4, scale=0.1, ptr=P, width=4, ws=P, out=None):
    pools = (ptr,) * (4 if fp8 else 2)
    fn = lib.pkv_tree_decode_fp8 if fp8 else lib.pkv_tree_decode
    out = ctypes.c_void_p(ptr.value + 4096) if ptr is not P and out is None else ptr
    return fn(ptr, *pools, ptr, width, ptr, ptr, ptr, words, batch, total, nodes, ctx, hq, hkv, d, bs, nb, scale, out, ws, 0, P)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_refuses(lib, fp8):
    assert attend(lib, fp8) == 1                                   # null pointers
    for bad in ({"batch": -1}, {"total": -1}, {"nodes": -1}, {"words": -1}, {"ctx": -1}, {"nb": 0}, {"width": 0}, {"scale": 0.0},
                {"scale": float("inf")}, {"scale": float("nan")}, {"nodes": 65}, {"nodes": 256, "words": 3}):
        assert attend(lib, fp8, ptr=X, **bad) == 1, bad
    for bad in ({"d": 64}, {"hq": 12, "hkv": 4}, {"bs": 100}, {"nodes": 257, "words": 5}, {"batch": 4097}, {"hq": 16, "hkv": 1},
                {"width": 1 << 23, "bs": 256}, {"ptr": ctypes.c_void_p(4104)}):
        assert attend(lib, fp8, **{"ptr": X, **bad}) == 2, bad
    assert attend(lib, fp8, ptr=X, ws=ctypes.c_void_p(4096 + 128)) == 3
    assert attend(lib, fp8, ptr=X, out=X) == 1                     # in place
    for none in ({"batch": 0}, {"total": 0}, {"nodes": 0}):
        assert attend(lib, fp8, **none) == 0, none


def test_workspace_size_refuses(lib):
    assert lib.pkv_tree_decode_workspace_size(4, 257, 16, 8, 128) == 0
    assert lib.pkv_tree_decode_workspace_size(4, 16, 12, 4, 128) == 0
    assert lib.pkv_tree_decode_workspace_size(-1, 16, 16, 8, 128) == 0


def test_accept_refuses(lib):
    def call(words=1, batch=2, total=10, nodes=9, path=4, ptr=X, new=ctypes.c_void_p(8192)):
        return lib.pkv_tree_accept(ptr, ptr, ptr, words, ptr, ptr, batch, total, nodes, path, ptr, ptr, ptr, new, P)
    assert call(ptr=P) == 1 and call(new=X) == 1                   # null; the lengths in place
    for bad in ({"batch": -1}, {"total": -1}, {"nodes": -1}, {"words": -1}, {"path": 0}, {"nodes": 65}):
        assert call(**bad) == 1, bad
    assert call(nodes=257, words=5) == 2
    assert call(batch=0, ptr=P) == 0


def pools(*addresses):
    return (ctypes.c_void_p * len(addresses))(*addresses)


def test_moves_refuse(lib):
    good, odd, null = pools(4096, 8192), pools(4096, 8200), pools(4096, None)

    def compact(k=good, v=good, ks=P, vs=P, layers=2, width=4, batch=2, path=4, nb=4, bs=256, hkv=8, d=128, ptr=X):
        return lib.pkv_tree_compact(k, v, ks, vs, layers, ptr, width, ptr, ptr, ptr, ptr, batch, path, nb, bs, hkv, d, P)

    def copy(k=good, v=good, ks=P, vs=P, layers=2, pairs=2, nb=4, bs=256, hkv=8, d=128, ptr=X):
        return lib.pkv_copy_blocks(k, v, ks, vs, layers, ptr, ptr, ptr, pairs, nb, bs, hkv, d, P)

    for call in (compact, copy):
        assert call(ptr=P) == 1
        for bad in ({"k": P}, {"v": null}, {"ks": good}, {"vs": good}, {"ks": good, "vs": null}, {"layers": -1}, {"nb": 0}, {"bs": 0}, {"hkv": 0}, {"d": 0}):
            assert call(**bad) == 1, bad
        for bad in ({"k": odd}, {"ks": good, "vs": odd}, {"layers": 129}, {"bs": 100}, {"d": 64}, {"hkv": 4097}):
            assert call(**bad) == 2, bad
        assert call(layers=0, k=P, v=P, ptr=P) == 0
    assert compact(batch=-1) == 1 and compact(path=-1) == 1 and compact(width=0) == 1 and compact(batch=65536) == 2
    assert compact(batch=0, ptr=P) == 0 and compact(path=0, ptr=P) == 0
    assert copy(pairs=-1) == 1 and copy(pairs=65536) == 2 and copy(pairs=0, ptr=P) == 0


def test_binding_refuses_cpu_tensors(lib):
    import paged_kv_attention_29_gb300 as pkv
    pool = torch.zeros(2, 256, 8, 128, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ids = torch.zeros(4, dtype=torch.int64)
    mask = torch.zeros(4, 1, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_tree_decode(torch.zeros(4, 16, 128, dtype=torch.bfloat16), pool, pool, i32(2, 1), i32(2), i32(3), mask, 4, 256, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_tree_accept(ids, ids, mask, i32(3), i32(2), 4, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.KvPools([pool], [pool])
    with pytest.raises(ValueError, match="one pool per layer"):
        pkv.KvPools([], [])
    with pytest.raises(ValueError, match="together"):
        pkv.KvPools([pool], [pool], k_scales=[pool])
