"""Filtered sampling on the GPU against the float64 oracle.

Ids must be the oracle's on every row whose outcome is decided by more than rounding: a race
margin above 1e-9 (near races are ranked in fp64) and a winner that does not change when top_p
moves by 1e-6 of itself (what the sums are good to).  Nearly every row is; each test bounds the others."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import filtered as fl
from pkv_testutil import expect_no_device_error

pytestmark = pytest.mark.gpu


def check(pkv, logits, T, k, p, m, seed=7, offset=0, most_unclear=1, view=None):
    B = logits.shape[0]
    t = lambda a, dt: torch.tensor(np.broadcast_to(a, (B,)).copy(), dtype=dt)  # noqa: E731
    T, k, p, m = t(T, torch.float32), t(k, torch.int32), t(p, torch.float32), t(m, torch.float32)
    ids = pkv.pkv_sample_filtered(logits.cuda() if view is None else view, T.cuda(), k.cuda(), p.cuda(), m.cuda(), seed, offset)
    ref, clear = fl.decided(logits.double().numpy(), T.double().numpy(), k.numpy(), p.double().numpy(), m.double().numpy(), seed, offset)
    got = ids.cpu().numpy()
    assert np.array_equal(got[clear], ref[clear]), (np.nonzero(clear & (got != ref))[0], got[got != ref], ref[got != ref])
    assert (~clear).sum() <= most_unclear
    expect_no_device_error(pkv)
    return got


def rows(B, V, seed, std=3.0, rounded=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, V, generator=g) * std
    return x.bfloat16().float() if rounded else x


SETTINGS = [(0, 1.0, 0.0), (1, 1.0, 0.0), (50, 1.0, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.05), (40, 0.8, 0.0), (100, 0.95, 0.01),
            (0, 0.3, 0.2), (10 ** 6, 0.999, 0.0), (2, 1e-6, 0.0)]


@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 31, 100, 1000, 4097])
@pytest.mark.parametrize("rounded", [False, True])
def test_small_rows_under_every_kind_of_filter(pkv, vocab, rounded):
    B = 4 * len(SETTINGS)
    k, p, m = (np.array(x * 4) for x in zip(*SETTINGS))
    T = np.random.default_rng(vocab).uniform(0.3, 1.5, B)
    check(pkv, rows(B, vocab, vocab + 1, 2.0, rounded), T, k, p, m, most_unclear=1)


@pytest.mark.parametrize("std,T", [(0.1, 1.0), (1.0, 1.0), (3.0, 0.7), (6.0, 0.3), (3.0, 5.0)])
def test_full_vocabulary_flat_to_peaked(pkv, std, T):
    """From rows on which top-p keeps most of the vocabulary (thousands of tokens share a bin) to
    rows with a few likely ones."""
    k, p, m = (np.array(x) for x in zip(*SETTINGS))
    check(pkv, rows(len(SETTINGS), W.VOCAB_QWEN3, 17, std), T, k, p, m)


def test_full_vocabulary_with_many_equal_logits(pkv):
    k = np.array([0, 1, 5, 900, 5000, 0, 0, 20000])
    p = np.array([0.5, 1.0, 0.9, 0.9, 0.7, 0.95, 0.1, 1.0])
    check(pkv, rows(8, W.VOCAB_QWEN3, 18, 1.0, True), 0.9, k, p, 0.0)
    check(pkv, torch.round(rows(8, 50000, 19, 1.0)), 0.9, k, p, 0.0)          # seven values in all
    flat = torch.zeros(8, 30011)                                              # one value: order by column alone
    check(pkv, flat, 1.0, k, p, 0.0)
    got = pkv.pkv_sample_filtered(flat.cuda(), torch.ones(8).cuda(), torch.full((8,), 1234, dtype=torch.int32).cuda(), None, None, 3)
    assert np.array_equal(got.cpu().numpy(), fl.sample(flat.numpy(), np.ones(8), np.full(8, 1234), np.ones(8), np.zeros(8), 3)[0])


def test_top_k_that_ends_in_the_far_tail(pkv):
    """Few likely tokens and a k that reaches far below them, with top-p on top of it."""
    x = rows(12, 20000, 20, 1.0) - 60
    x[:, 100:103] = torch.tensor([5.0, 4.0, 3.0])
    check(pkv, x, 1.0, np.array([2, 3, 4, 10, 3000, 19999] * 2), np.array([0.99999] * 6 + [1.0] * 6), 0.0)
    check(pkv, x, 0.05, np.array([2, 3, 4, 10, 3000, 19999] * 2), np.array([0.9] * 6 + [1.0] * 6), 0.0)


def test_masked_infinite_and_nan_logits(pkv):
    x = rows(16, 3001, 21)
    g = torch.Generator().manual_seed(22)
    x[torch.rand(x.shape, generator=g) < 0.8] = -float("inf")
    x[torch.rand(x.shape, generator=g) < 0.05] = float("nan")
    x[0] = -float("inf")
    x[1] = float("nan")
    x[2] = -float("inf")
    x[2, 77] = -1e30
    x[3, 500] = x[3, 40] = float("inf")
    x[4, 3000] = float("inf")
    x[5] = torch.finfo(torch.float32).min
    x[5, 9] = -3e38
    ids = check(pkv, x, 0.8, np.array([0, 5] * 8), np.array([1.0, 0.9, 0.5, 1.0] * 4), np.array([0.0] * 8 + [0.1] * 8))
    assert ids[:6].tolist()[:5] == [-1, -1, 77, 40, 3000] and ids[5] == 9


def test_all_off_is_the_plain_sampler(pkv):
    s = W.sampler_inputs(batch=64, vocab=30001, seed=23, device="cpu")
    x, T = s.logits.cuda(), s.temperatures.cuda()
    ref = pkv.pkv_sample(x, T, s.seed, 12345678901)
    assert torch.equal(ref, pkv.pkv_sample_filtered(x, T, None, None, None, s.seed, 12345678901))
    off = torch.zeros(64, dtype=torch.int32).cuda(), torch.ones(64).cuda(), torch.zeros(64).cuda()
    assert torch.equal(ref, pkv.pkv_sample_filtered(x, T, *off, s.seed, 12345678901))
    assert torch.equal(ref, pkv.pkv_sample_filtered_dev(x, T, None, None, None, torch.tensor([s.seed, 12345678901]).cuda()))


def test_strided_and_unaligned_rows(pkv):
    x = rows(9, 3000, 24)
    wide = torch.full((9, 3010), 99.0)
    wide[:, 1:3001] = x
    k, p = np.array([0, 20, 0] * 3), np.array([1.0, 0.9, 0.6] * 3)
    check(pkv, x, 0.9, k, p, 0.0, view=wide.cuda()[:, 1:3001])
    check(pkv, x[:1], 0.9, k[1:2], p[1:2], 0.0, view=wide.cuda()[:1, 1:3001])


def test_a_vocabulary_larger_than_shared_memory(pkv):
    x = rows(4, 250001, 25, 2.0)
    check(pkv, x, 0.8, np.array([0, 50, 0, 2000]), np.array([0.9, 1.0, 1.0, 0.8]), np.array([0.0, 0.0, 0.05, 0.0]))


def test_extreme_temperatures(pkv):
    x = rows(6, 500, 26)
    check(pkv, x, np.array([1e-30, 1e-6, 1e-3, 50.0, 1e6, 1e30]), np.array([0, 5, 0, 0, 30, 0]), np.array([0.9, 1.0, 0.5, 0.5, 0.7, 0.25]), 0.0)


def test_near_ties_are_ranked_in_fp64(pkv):
    """Rows built so that the two best keys are 1e-6 apart, closer than fp32 keys can tell."""
    from oracle import sampler as sm
    V, seed = 4096, 31
    e = sm.exponential_noise(seed, 0, range(32), V)
    x = torch.full((32, V), -50.0)
    for b in range(32):
        i, j = 100 + 7 * b, 3000 - 11 * b
        x[b, i] = 1.0
        want = 1.0 - np.log(e[b, i]) + np.log(e[b, j]) + (1e-6 if b % 2 else -1e-6)
        x[b, j] = float(np.float32(want))
    check(pkv, x, 1.0, 0, 1.0, 0.0, seed=seed)
    check(pkv, x, 1.0, 2, 1.0, 0.0, seed=seed)


def test_refused_rows_are_flagged_and_the_others_run(pkv):
    x = rows(6, 100, 27).cuda()
    T = torch.ones(6).cuda()
    ok = pkv.pkv_sample_filtered(x, T, None, None, None, 1)
    for name, bad in (("p", 0.0), ("p", -0.1), ("p", 1.5), ("p", float("nan")), ("m", -0.1), ("m", 1.1), ("m", float("nan"))):
        f = torch.full((6,), 1.0 if name == "p" else 0.0)
        f[4] = bad
        ids = pkv.pkv_sample_filtered(x, T, None, f.cuda() if name == "p" else None, f.cuda() if name == "m" else None, 1)
        assert pkv.pkv_get_device_error(clear=True) == (8, 4)
        assert ids[4] == -1 and torch.equal(ids[[0, 1, 2, 3, 5]], ok[[0, 1, 2, 3, 5]])
    T[2] = 0.0
    ids = pkv.pkv_sample_filtered(x, T, None, None, None, 1)
    assert pkv.pkv_get_device_error(clear=True) == (4, 2) and ids[2] == -1
    for wrong in (dict(top_k=torch.zeros(5, dtype=torch.int32).cuda()), dict(top_k=torch.zeros(6, dtype=torch.int64).cuda()),
                  dict(top_p=torch.ones(6, dtype=torch.float64).cuda()), dict(min_p=torch.zeros(6))):
        with pytest.raises((TypeError, ValueError)):
            pkv.pkv_sample_filtered(x, T, wrong.get("top_k"), wrong.get("top_p"), wrong.get("min_p"), 1)


def test_frequencies_follow_the_filtered_distribution(pkv):
    """Many rows of one distribution: top-p 0.75 of (0.4, 0.3, 0.2, 0.1) keeps three, renormalised."""
    n = 20000
    x = torch.log(torch.tensor([0.1, 0.3, 0.2, 0.4])).expand(n, 4).contiguous().cuda()
    ids = pkv.pkv_sample_filtered(x, torch.ones(n).cuda(), None, torch.full((n,), 0.75).cuda(), None, seed=5)
    freq = np.bincount(ids.cpu().numpy(), minlength=4) / n
    want = np.array([0.0, 3, 2, 4]) / 9
    assert np.all(np.abs(freq - want) <= 4 * np.sqrt(want * (1 - want) / n))


def test_captured_with_fresh_noise_and_settings(pkv):
    x = rows(32, 5003, 28)
    gx, T = x.cuda(), torch.full((32,), 0.8).cuda()
    k, p, m = torch.full((32,), 30, dtype=torch.int32).cuda(), torch.full((32,), 0.9).cuda(), torch.zeros(32).cuda()
    so, ids = torch.tensor([3, 0]).cuda(), torch.empty(32, dtype=torch.int64).cuda()
    run = lambda: pkv.pkv_sample_filtered_dev(gx, T, k, p, m, so, out_ids=ids)  # noqa: E731
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for step in range(3):
        so.copy_(torch.tensor([3, 32 * step]))
        k.fill_(30 - 10 * step)
        p.fill_(0.9 - 0.2 * step)
        graph.replay()
        assert torch.equal(ids, pkv.pkv_sample_filtered(gx, T, k, p, m, 3, 32 * step))
    check(pkv, x, 0.8, 10, np.float32(0.5), 0.0, seed=3, offset=64)


@pytest.mark.parametrize("B,vocab", [(9, 3001), (77, 12007), (160, 30011), (300, 129)])
def test_batches_of_every_size(pkv, B, vocab):
    """Few, some and many rows run as clusters of different sizes; every kind of row in each."""
    k, p, m = (np.array([SETTINGS[i % len(SETTINGS)][j] for i in range(B)]) for j in range(3))
    T = np.random.default_rng(B).uniform(0.4, 1.3, B)
    check(pkv, rows(B, vocab, B + 3, 2.5, rounded=B % 2 == 0), T, k, p, m, most_unclear=2)


def test_many_rows_of_a_vocabulary_beyond_the_lists(pkv):
    """Slices too long for the warps' lists of quads are walked instead."""
    B = 80
    x = rows(B, 180001, 41, 2.0)
    k, p = np.where(np.arange(B) % 4 == 0, 30, 0), np.where(np.arange(B) % 4 == 1, 1.0, 0.85)
    check(pkv, x, 0.9, k, p, 0.0, most_unclear=2)


@pytest.mark.parametrize("vocab", [5, 1001, 30011])
def test_one_row_of_an_odd_vocabulary(pkv, vocab):
    for i, (k, p, m) in enumerate(SETTINGS):
        check(pkv, rows(1, vocab, 60 + i), 0.8, k, p, m)


@pytest.mark.parametrize("B", [8, 400])
def test_top_p_borders_anywhere_in_a_row(pkv, B):
    """One row under many p, so that borders lie in every part of the order, on histogram bins' and
    threads' limits too."""
    x = rows(1, 20011, 71, 1.5)
    p = np.linspace(0.0005, 0.9995, 400)
    for i in range(0, 400, B):
        check(pkv, x.expand(B, -1).contiguous(), 0.9, 0, p[i:i + B], 0.0, offset=i)


@pytest.mark.parametrize("B", [40, 200])
def test_full_vocabulary_in_larger_batches(pkv, B):
    """Rows of one batch from flat to peaked, with settings that end a row in each of its ways: a race's
    winner that stands, one that does not with few or with many tokens before it, a border looked for."""
    x = rows(B, W.VOCAB_QWEN3, 81, 1.0) * torch.logspace(-2, 1, B)[torch.randperm(B, generator=torch.Generator().manual_seed(82))][:, None]
    more = SETTINGS + [(0, 0.02, 0.0), (0, 0.5, 0.0), (0, 0.5, 0.02), (1000, 0.7, 0.0), (300, 1.0, 0.0)]
    k, p, m = (np.array([more[i % len(more)][j] for i in range(B)]) for j in range(3))
    check(pkv, x, np.random.default_rng(83).uniform(0.4, 1.5, B), k, p, m, most_unclear=3)


@pytest.mark.parametrize("B", [1000, 4097])
def test_every_row_of_a_large_batch_is_sampled(pkv, B):
    """Batches whose rows do not all run at once take them in another order than the rows'."""
    rng = np.random.default_rng(B)
    k, p, m = (np.array([SETTINGS[i][j] for i in rng.integers(0, len(SETTINGS), B)]) for j in range(3))
    check(pkv, rows(B, 129, 91), 0.9, k, p, m, most_unclear=5)
