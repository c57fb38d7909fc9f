"""How near to a border of top-p a token is still decided as in exact arithmetic.

Each row has one token that would win any race (the best noise, in a row whose other good noise belongs to its
lowest logits), and a top_p for which the weights before that token are 1.5e-6 of themselves on one side or the other of
the border; weights and sums are good to about 1e-6.  The batches are of the three sizes whose threads sum the
smallest and the largest shares of a row, at a vocabulary of 200,000."""
import numpy as np
import pytest
import torch

from oracle import sampler as sm
from pkv_testutil import expect_no_device_error

V, T, SLACK = 200000, np.float32(0.9), 1.5e-6
VALUES = {
    "nearly flat": lambda r: -0.05 * r.random(V),
    "spread": lambda r: -3.0 * r.random(V),
    "normal": lambda r: r.normal(size=V),
    "wide": lambda r: 2.0 * r.normal(size=V),
    "steps": lambda r: -0.3 * r.integers(0, 8, V),
}


def border_row(kind, seed, row):
    """(logits, top_p, the token, whether it is in)."""
    rng = np.random.default_rng(100 * seed + row)
    g = -np.log(sm.exponential_noise(seed, 0, [row], V)[0])
    by_noise = np.argsort(g, kind="stable")
    token = int(by_noise[-1])
    values = -np.sort(-VALUES[kind](rng).astype(np.float32))
    at = int(rng.uniform(0.05, 0.9) * V)
    x = np.empty(V, np.float32)
    x[token] = values[at]
    x[by_noise[:-1]] = np.delete(values, at)
    order = np.lexsort((np.arange(V), -x))
    w = np.exp((x[order].astype(np.float64) - x[order[0]]) / float(T))
    before = (np.cumsum(w) - w)[int(np.nonzero(order == token)[0][0])]
    p = np.float32(before / w.sum() / (1 + (SLACK if row % 2 else -SLACK)))
    off = before / (float(p) * w.sum()) - 1
    assert abs(off) > SLACK - 2.0 ** -23                  # top_p's own rounding
    key = (x.astype(np.float64) - x.max()) / float(T) + g
    assert key.argmax() == token
    return x, p, token, off < 0


def test_the_rows_are_what_they_are_meant_to_be():
    for i, kind in enumerate(VALUES):
        assert [border_row(kind, 5, row)[3] for row in (2 * i, 2 * i + 1)] == [True, False]


@pytest.mark.gpu
@pytest.mark.parametrize("B", [6, 24, 192])
@pytest.mark.parametrize("kind", VALUES)
def test_tokens_at_a_border_of_top_p(pkv, kind, B):
    n = min(B, 12)
    x, p = torch.zeros(B, V), np.full(B, 0.5, np.float32)
    token, inside = np.zeros(n, np.int64), np.zeros(n, bool)
    for b in range(n):
        row, p[b], token[b], inside[b] = border_row(kind, 5, b)
        x[b] = torch.from_numpy(row)
    ids = pkv.pkv_sample_filtered(x.cuda(), torch.full((B,), float(T)).cuda(), None, torch.from_numpy(p).cuda(), None, 5)
    assert np.array_equal(ids[:n].cpu().numpy() == token, inside)
    expect_no_device_error(pkv)
