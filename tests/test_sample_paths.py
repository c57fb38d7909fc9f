"""Filtered sampling on the ways through its kernel that ordinary rows hardly ever take.

Most rows without top-k end at a race's winner.  The rows built here do not: their noise is known, so the tokens
that win their races are made the last in the order of logits, far outside top-p, and the kernel has to look for
the border itself.  Which way a row takes is replayed here from the kernel's own constants, so that a later
change of those cannot quietly lead the rows past what they are for; the replays run without a GPU."""
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_attention_29_gb300 as package
from oracle import filtered as fl
from oracle import sampler as sm
from pkv_testutil import expect_no_device_error

SOURCE = open(os.path.join(os.path.dirname(package.__file__), "csrc", "sample_filtered.cu")).read()


def constant(name):
    return float(re.search(rf"constexpr \w+ {name} = ([\d.]+)f?;", SOURCE).group(1))


BINS, CAP, BORDER, LISTED, TRIES, CANDS, WIDE = (int(constant(c)) for c in
                                                 ("BINS", "CAP", "BORDER", "LISTED", "TRIES", "CANDS", "kWideRows"))
BINS_PER_OCTAVE = constant("BINS_PER_OCTAVE")
SHAPES = {name: tuple(v.strip() for v in body.split(","))
          for name, body in re.findall(r"using (\w+Rows) = Rows<([^>]*)>;", SOURCE)}


def shape_of(batch, sms):
    """(clusters' CTAs, threads, candidates of a race) of a batch."""
    name = "FewRows" if batch <= WIDE else "SomeRows" if 4 * batch <= 5 * sms else "ManyRows"
    cluster, threads, _, _, tried = SHAPES[name]
    return name, int(cluster), int(threads), CANDS if tried == "CANDS" else int(tried)


def longest_listed(cluster, threads):
    """Logits of the longest row whose slices fit the warps' lists."""
    return LISTED // (threads // 32) // 32 * threads * cluster * 4


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152


def row_of(values, seed, row):
    """These values as one row of logits: the better a column's noise, the lower its logit."""
    g = -np.log(sm.exponential_noise(seed, 0, [row], len(values))[0])
    x = np.empty(len(values), np.float32)
    x[np.argsort(g, kind="stable")] = -np.sort(-values.astype(np.float32), kind="stable")
    return x


def way(x, T, p, min_p, seed, row, tried):
    """How the kernel ends a row without top-k: "race" by a winner that stands, "list" on the few tokens before
    one that does not, or "border"; with the members of the bins that the border can lie in (about: the bins
    of 1/64 octave that hold the last kept token and the first left out), and the largest number of equal logits there."""
    order = np.lexsort((np.arange(len(x)), -x))
    z = (x[order].astype(np.float64) - x[order[0]]) / T
    w = np.exp(z)
    before = np.cumsum(w) - w
    n = int(np.searchsorted(before, p * w.sum(), side="left"))
    key = z - np.log(sm.exponential_noise(seed, 0, [row], len(x))[0][order])
    if min_p > 0:
        key[z < np.log(min_p)] = -np.inf
    left = len(x)
    end = None
    for _ in range(TRIES):
        best = np.argsort(-key[:left], kind="stable")[:tried]
        best = best[key[best] > -np.inf]
        if (best < n).any():
            end = "race"
            break
        left = int(best.min())
        if left <= CAP:
            end = "list"
            break
    bins = (-z * np.log2(np.e) * BINS_PER_OCTAVE).astype(np.int64)
    near = (bins >= bins[n - 1]) & (bins <= bins[min(n, len(x) - 1)])
    equal = int(np.unique(x[order][near], return_counts=True)[1].max())
    return end or "border", int(near.sum()), equal


V = 20000


def tail(size):
    """Of a row's values, the last ones: each lower than the one before it."""
    return -0.0005 * np.maximum(0, np.arange(V) - (V - size))


# what the row's values are like, top-p, min-p: and what that makes of the border
LATE = {
    "spread": (lambda r: -3.0 * r.random(V), 0.4, 0.0),                        # few members in a bin
    "spread, far": (lambda r: -3.0 * r.random(V), 0.85, 0.0),
    "nearly flat": (lambda r: -0.05 * r.random(V), 0.3, 0.0),                  # thousands in a bin: the second histogram
    "nearly flat, early": (lambda r: -0.02 * r.random(V), 0.15, 0.0),
    "steps of hundreds": (lambda r: -0.02 * r.integers(0, 30, V), 0.5, 0.0),   # equal logits at the border, halved or collected
    "steps of thousands": (lambda r: -0.5 * r.integers(0, 6, V), 0.6, 0.0),
    "flat": (lambda r: tail(1000), 0.25, 0.0),                                 # one value and a tail: the order is the columns'
    "flat with min-p": (lambda r: tail(200) - 0.3 * (np.arange(V) > 9000), 0.6, 0.5),
    "spread with min-p": (lambda r: -2.0 * r.random(V), 0.45, 0.13),
    "steps with min-p": (lambda r: -0.25 * r.integers(0, 8, V), 0.4, 0.15),
}


def late_row(kind, seed, row):
    values, p, m = LATE[kind]
    return row_of(values(np.random.default_rng(1000 * seed + row)), seed, row), np.float32(p), np.float32(m)


@pytest.mark.parametrize("tried", sorted({shape_of(b, 152)[3] for b in (3, 40, 200)}))
@pytest.mark.parametrize("kind", LATE)
def test_the_rows_below_reach_the_border(kind, tried):
    for row in (0, 5):
        x, p, m = late_row(kind, 11, row)
        end, members, equal = way(x, 0.9, float(p), float(m), 11, row, tried)
        assert end == "border"
        if kind.startswith("spread"):
            assert members <= BORDER
        if kind.startswith("nearly flat"):
            assert members > BORDER and equal <= 2
        if kind == "steps of hundreds":
            assert BORDER < equal < CAP
        if kind in ("steps of thousands", "flat", "flat with min-p"):
            assert equal > CAP


def check_rows(pkv, x, T, k, p, m, seed, rows):
    """Ids of a batch; the given rows against the oracle."""
    B = len(x)
    f = lambda a, dt: np.broadcast_to(np.asarray(a, dt), (B,)).copy()  # noqa: E731
    T, k, p, m = f(T, np.float32), f(k, np.int32), f(p, np.float32), f(m, np.float32)
    ids = pkv.pkv_sample_filtered(x.cuda(), *(torch.from_numpy(a).cuda() for a in (T, k, p, m)), seed).cpu().numpy()
    expect_no_device_error(pkv)
    unclear = 0
    for b in rows:
        ref, clear = fl.decided(x[b:b + 1].double().numpy(), T[b:b + 1].astype(float), k[b:b + 1], p[b:b + 1].astype(float),
                                m[b:b + 1].astype(float), seed, b)
        unclear += int(not clear[0])
        assert not clear[0] or ids[b] == ref[0], (b, ids[b], ref[0], k[b], p[b], m[b])
    assert unclear <= 1 + len(list(rows)) // 10
    return ids


@pytest.mark.gpu
@pytest.mark.parametrize("B", [5, 40, 200])
def test_borders_are_found_by_every_shape_of_cluster(pkv, B):
    _, _, _, tried = shape_of(B, sms())
    assert [shape_of(b, sms())[0] for b in (5, 40, 200)] == ["FewRows", "SomeRows", "ManyRows"]
    kinds = list(LATE)
    for seed in range(12, 12 + (2 if B > 5 else 4)):
        x, p, m = (np.stack(a) for a in zip(*(late_row(kinds[(b + seed * 5) % len(kinds)], seed, b) for b in range(B))))
        rows = list(range(min(B, 30))) + list(range(B - 10, B)) * (B > 40)
        ways = [way(x[b], 0.9, float(p[b]), float(m[b]), seed, b, tried)[0] for b in rows]
        assert ways.count("border") >= 0.9 * len(rows)
        check_rows(pkv, torch.from_numpy(x), 0.9, 0, p, m, seed, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [5, 40, 200])
def test_large_k_in_every_shape_of_cluster(pkv, B):
    """More than the threads can bound (k above 1024), thousands of equal logits at the k-th, and a bound that
    more tokens reach than fit the list; with top-p and min-p on top."""
    g = torch.Generator().manual_seed(B)
    x = torch.randn(B, V, generator=g)
    x[1::4] = torch.round(x[1::4] * 2) / 2
    x[2::4] *= 0.01
    x[3::4] = torch.round(x[3::4])
    r = np.arange(B)
    k = np.array([1500, 3000, 50, 9000, 1025, 5000, 400])[r % 7]
    p = np.array([1.0, 0.7, 0.95, 0.3, 1.0])[r % 5]
    m = np.array([0.0, 0.0, 0.02])[r % 3]
    check_rows(pkv, x, 0.8, k, p, m, 21, list(range(min(B, 35))) + list(range(B - 8, B)) * (B > 40))


@pytest.mark.gpu
@pytest.mark.parametrize("B,over", [(2, 44641), (12, 2321), (200, 16161)])
def test_slices_beyond_the_warps_lists(pkv, B, over):
    """Rows too long for the lists of quads are walked instead: races under min-p, borders of top-p (with and without
    a second histogram, and with thousands of equal logits), a large k with top-p."""
    _, cluster, threads, tried = shape_of(B, sms())
    vocab = longest_listed(cluster, threads) + over
    rows = list(range(min(B, 12)))
    g = torch.Generator().manual_seed(B)
    for first in range(0, 12 if B == 2 else 1, B):
        x = torch.randn(B, vocab, generator=g) * 2
        k, p, m = np.zeros(B, np.int32), np.ones(B, np.float32), np.zeros(B, np.float32)
        for b in range(B):
            i = (first + b) % 12
            rng = np.random.default_rng(100 * i + B)
            if b >= 12:
                p[b], m[b] = (0.9, 0.0) if b % 2 else (1.0, 0.05)
            elif i < 4:                                   # late winners
                values = (-3.0 * rng.random(vocab), -0.05 * rng.random(vocab), -0.5 * rng.integers(0, 6, vocab),
                          -0.0005 * np.maximum(0, np.arange(vocab) - (vocab - 1000)))[i]
                x[b] = torch.from_numpy(row_of(values, 31, b))
                p[b] = (0.4, 0.3, 0.6, 0.25)[i]
                assert way(x[b].numpy(), 0.9, float(p[b]), 0.0, 31, b, tried)[0] == "border"
            else:
                k[b], p[b], m[b] = ((0, 1.0, 0.05), (0, 0.9, 0.01), (2000, 0.8, 0.0), (50, 1.0, 0.0), (0, 0.5, 0.2), (30000, 0.95, 0.02),
                                    (0, 1.0, 0.0), (0, 0.999, 0.0))[i - 4]
        check_rows(pkv, x, 0.9, k, p, m, 31, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("B,vocab", [(5, 7), (40, 3001), (200, 3001), (200, 5)])
def test_masks_of_the_lowest_finite_value(pkv, B, vocab):
    """A row that holds nothing but the lowest finite value is a flat row; beside other logits such tokens weigh
    nothing, like ones at -inf."""
    r = np.arange(B)
    lowest = torch.finfo(torch.float32).min
    T = torch.from_numpy(np.array([0.05, 0.9, 3.0], np.float32)[r % 3]).cuda()
    k = torch.from_numpy(np.array([0, 0, 2, 3, 1025], np.int32)[r % 5]).cuda()
    p = torch.from_numpy(np.array([1.0, 0.9, 0.5, 1e-6], np.float32)[r % 4]).cuda()
    m = torch.from_numpy(np.array([0.0, 0.0, 0.2], np.float32)[r // 2 % 3]).cuda()
    flat = torch.zeros(B, vocab, device="cuda")
    args = (T, k, p, m, 51)
    assert torch.equal(pkv.pkv_sample_filtered(flat, *args), pkv.pkv_sample_filtered(flat + lowest, *args))
    g = torch.Generator().manual_seed(52)
    x = torch.randn(B, vocab, generator=g) * 2
    out = torch.rand(B, vocab, generator=g) < 0.9
    out[r, r % vocab] = False
    args = (T, k, p, m, 53)
    a, b = (pkv.pkv_sample_filtered(x.masked_fill(out, v).cuda(), *args) for v in (lowest, -float("inf")))
    assert torch.equal(a, b)
    expect_no_device_error(pkv)
