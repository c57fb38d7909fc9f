"""The 8-bit cache's and the filters' oracles against closed forms, torch's own conversion and
brute force; the host checks of the new entry points (no GPU)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from oracle import filtered as fl
from oracle import fp8_cache as fc
from oracle import sampler as sm


def test_e4m3_table_is_the_format():
    ours = fc.E4M3
    theirs = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(ours), np.isnan(theirs)) and np.isnan(ours).sum() == 2
    assert np.array_equal(ours[~np.isnan(ours)], theirs[~np.isnan(theirs)])
    assert ours[126] == 448 and ours[1] == 2.0 ** -9


def test_rounding_matches_torch_and_ties_go_to_even():
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(4000, generator=g) * 50, torch.randn(4000, generator=g) * 2.0 ** -8,
                   torch.tensor([0.0, -0.0, 448.0, -448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])]).clamp(-448, 448)
    ours = fc.round_e4m3(x.double().numpy())
    theirs = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ours, theirs)
    # 17 lies between 16 (code even) and 18, 19 between 18 and 20 (even)
    assert fc.E4M3[fc.round_e4m3(17.0)] == 16 and fc.E4M3[fc.round_e4m3(19.0)] == 20


def test_scale_is_the_smallest_that_fits():
    for amax, e in ((448.0, 0), (449.0, 1), (1.0, -8), (0.875, -9), (0.876, -8), (0.0, -126), (2.0 ** -140, -126),
                    (3.3e38, 120)):
        assert fc.scale_exponent(amax) == e, amax
    codes, s = fc.quantise_rows(np.array([[448.0, -1.0], [np.inf, 1.0], [np.nan, 1.0], [0.0, 0.0]]))
    assert s.tolist() == [127, 255, 255, 1] and codes[1].tolist() == [0, 0]
    read = fc.read_rows(codes, s)
    assert read[0].tolist() == [448.0, -1.0] and np.isnan(read[1]).all() and np.isnan(read[2]).all() and not read[3].any()


def test_read_is_within_half_a_step():
    x = np.random.default_rng(2).normal(size=(200, 128)) * np.exp2(np.random.default_rng(3).integers(-20, 20, (200, 1)))
    codes, s = fc.quantise_rows(x)
    e = s.astype(int) - 127
    assert np.all(np.abs(fc.read_rows(codes, s) - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** (e - 10.0)[:, None])
    amax = np.abs(x).max(1)
    assert np.all(amax <= 448 * 2.0 ** e) and np.all(amax > 448 * 2.0 ** (e - 1.0))


def test_store_scatters_rows_and_scales():
    rng = np.random.default_rng(4)
    codes, scales = rng.integers(0, 120, (3, 4, 2, 8), dtype=np.uint8), rng.integers(100, 140, (3, 2, 4), dtype=np.uint8)
    x = rng.normal(size=(3, 2, 8))
    c2, s2 = fc.store(codes, scales, x, [9, -1, 2])
    qc, qs = fc.quantise_rows(x)
    assert np.array_equal(c2[2, 1], qc[0]) and np.array_equal(s2[2, :, 1], qs[0])
    assert np.array_equal(c2[0, 2], qc[2]) and np.array_equal(s2[0, :, 2], qs[2])
    same = np.ones((3, 4), bool)
    same[2, 1] = same[0, 2] = False
    assert np.array_equal(c2[same], codes[same]) and np.array_equal(s2.swapaxes(1, 2)[same], scales.swapaxes(1, 2)[same])


def test_kept_by_brute_force():
    """kept() against the definition walked token by token, on rows with ties and masked tokens."""
    rng = np.random.default_rng(5)
    for k, p, m in itertools.product((0, 1, 3, 100), (1.0, 0.9, 0.3, 1e-6), (0.0, 0.1, 1.0)):
        l = np.round(rng.normal(size=12) * 2) / 2
        l[rng.integers(0, 12, 3)] = -np.inf
        T = 0.7
        todo = sorted((v for v in range(12) if l[v] > -np.inf), key=lambda v: (-l[v], v))
        top = todo[:k] if k else todo
        w = {v: np.exp((l[v] - l[todo[0]]) / T) for v in top}
        out, before = [], 0.0
        for v in top:
            if p >= 1 or before < p * sum(w.values()):
                out.append(v)
            before += w[v]
        out = [v for v in out if w[v] >= m * (1 - 1e-12)]
        assert fl.kept(l, T, k, p, m).tolist() == out, (k, p, m)


def test_filters_off_is_the_plain_race_and_k1_is_the_maximum():
    rng = np.random.default_rng(6)
    l = rng.normal(size=(40, 300)) * 3
    T = rng.uniform(0.5, 1, 40)
    off = np.zeros(40), np.ones(40), np.zeros(40)
    assert np.array_equal(fl.sample(l, T, *off, 9, 4)[0], sm.sample(l, T, 9, 4)[0])
    assert np.array_equal(fl.sample(l, T, np.ones(40), *off[1:], 9, 4)[0], l.argmax(1))
    assert np.array_equal(fl.sample(l, T, off[0], np.full(40, 1e-9), off[2], 9, 4)[0], l.argmax(1))
    assert np.array_equal(fl.sample(l, T, off[0], off[1], np.ones(40), 9, 4)[0], l.argmax(1))


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_29_gb300 import build
    build.build()
    import paged_kv_attention_29_gb300 as pkv
    return pkv.load()


def test_refusals_come_before_any_launch(lib):
    P = None
    at = ctypes.c_void_p(256)                # non-null and aligned, never dereferenced: the check returns first
    odd = ctypes.c_void_p(8)
    store = lambda k=P, n=4, ks=1024, vs=1024, nb=4, bs=256, hkv=8, d=128, pool=P, sc=P: lib.pkv_store_kvcache_fp8(  # noqa: E731
        k, k, n, ks, vs, k, pool, pool, sc, sc, nb, bs, hkv, d, P)
    assert store() == 1 and store(n=-1) == 1 and store(ks=512) == 1 and store(vs=512) == 1 and store(n=0) == 0
    assert store(d=64, ks=1024) == 2 and store(bs=100) == 2 and store(hkv=0) == 1 and store(nb=0) == 1
    assert store(k=at, pool=at, sc=P) == 1                       # no scale pools
    assert store(k=at, pool=odd, sc=at) == 2 and store(k=at, pool=at, sc=odd) == 2 and store(k=odd, pool=at, sc=at) == 2
    assert store(k=at, pool=at, sc=at, ks=1028) == 2             # stride not a multiple of 8
    rope = lambda q=P, qo=P, qs=0, qos=0, k=P, pos=P, n=4, hq=0, base=1e4, d=128, bs=256: lib.pkv_rope_store_kvcache_fp8(  # noqa: E731
        q, qs, qo, qos, k, 1024, k, 1024, pos, n, hq, 8, d, base, k, k, k, k, k, 4, bs, P)
    assert rope() == 1 and rope(n=0) == 0 and rope(base=0.0) == 1 and rope(base=float("nan")) == 1 and rope(base=float("inf")) == 1
    assert rope(q=at, qs=2048, hq=16) == 1                       # q without q_out
    assert rope(q=at, qo=at, qs=2048, qos=4096, hq=16) == 1      # in place with other strides
    assert rope(q=at, qo=at, qs=2048, qos=2048, hq=0) == 1 and rope(q=at, qo=at, qs=100, qos=2048, hq=16) == 1
    assert rope(k=at) == 1                                       # no positions
    assert rope(d=64) == 2 and rope(bs=128) == 2
    dec = lambda ptr=P, mb=4, b=2, hq=16, hkv=8, d=128, bs=256, nb=4, sc=0.1, ws=P, n=0: lib.pkv_decode_fp8(  # noqa: E731
        ptr, ptr, ptr, ptr, ptr, ptr, mb, ptr, b, 10, hq, hkv, d, bs, nb, sc, ptr, ws, n, P)
    assert dec() == 1 and dec(b=0) == 0 and dec(b=-1) == 1 and dec(mb=0) == 1 and dec(nb=0) == 1
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert dec(sc=bad) == 1
    assert dec(hq=12, hkv=4) == 2 and dec(hq=16, hkv=1) == 2 and dec(d=64) == 2 and dec(bs=100) == 2
    assert dec(mb=2 ** 24) == 2                                  # positions beyond 32 bits
    assert dec(ptr=odd) == 2 and dec(ptr=at, ws=odd) == 3
    assert lib.pkv_decode_fp8_workspace_size(4, 12, 4, 128) == 0 and lib.pkv_decode_fp8_workspace_size(-1, 16, 8, 128) == 0
    pre = lambda ptr=P, mb=4, ns=2, tq=10, mq=9, mk=9, tk=20, hq=16, hkv=8, d=128, bs=256, nb=4, sc=0.1, ws=P: lib.pkv_prefill_varlen_fp8(  # noqa: E731
        ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, mb, ns, tq, mq, mk, tk, hq, hkv, d, bs, nb, sc, ptr, ws, 0, P)
    assert pre() == 1 and pre(ns=0) == 0 and pre(tq=0) == 0 and pre(mk=8) == 1 and pre(tk=-1) == 1 and pre(ns=-1) == 1
    assert pre(sc=0.0) == 1 and pre(sc=float("nan")) == 1 and pre(hq=12, hkv=4) == 2 and pre(d=64) == 2 and pre(bs=128) == 2
    assert pre(ptr=odd) == 2 and pre(ptr=at, ws=odd) == 3 and pre(ptr=at, ns=70000) == 2 and pre(ptr=at, tk=2 ** 40) == 2
    size = lib.pkv_prefill_fp8_workspace_size
    assert size(2, 16, 8, 128, 9, 9, 20) >= 2 * 20 * 8 * 128 * 2 and size(2, 12, 4, 128, 9, 9, 20) == 0
    assert size(2, 16, 8, 128, 9, 9, -1) == 0 and size(2, 16, 8, 128, -1, 9, 20) == 0
    smp = lambda ptr=P, b=2, v=100, st=100: lib.pkv_sample_filtered(ptr, b, v, st, ptr, P, P, P, 0, 0, ptr, P)  # noqa: E731
    assert smp() == 1 and smp(b=0) == 0 and smp(v=0, st=0) == 1 and smp(st=50) == 1 and smp(b=-1) == 1
    assert smp(ptr=at, b=70000) == 2 and smp(ptr=at, v=2 ** 24 + 1, st=2 ** 25) == 2
    dev = lambda so: lib.pkv_sample_filtered_dev(at, 2, 100, 100, at, P, P, P, so, at, P)  # noqa: E731
    assert dev(P) == 1 and dev(ctypes.c_void_p(12)) == 1


def test_binding_refuses_wrong_tensors(lib):
    import paged_kv_attention_29_gb300 as pkv
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(2, 256, 8, 128).to(torch.float8_e4m3fn)
    sc = torch.zeros(2, 8, 256, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    i4 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_store_kvcache_fp8(x, x, i4, pool, pool, sc, sc)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_decode_fp8(x, pool, pool, sc, sc, i4.view(4, 1), i4, 1, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_sample_filtered(torch.zeros(4, 9), torch.ones(4), None, None, None, seed=1)
