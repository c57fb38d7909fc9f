"""min-p's limit, at the logits' own resolution.

A row keeps z = (logit - largest) / T >= ln(min_p).  The rows here hold one token on each side of that limit, one
step of their logits apart, at magnitudes where a step is far above the limit's own precision of 2^-22 of itself."""
import numpy as np
import pytest
import torch

from oracle import filtered as fl
from oracle import sampler as sm
from pkv_testutil import expect_no_device_error


def cut_rows(B, seed):
    """Rows whose two best-placed tokens lie just below and just above min-p's limit, by one step of their logits."""
    V, rng = 1024, np.random.default_rng(seed)
    g = -np.log(sm.exponential_noise(seed, 0, range(B), V))
    x = np.full((B, V), -np.inf, np.float32)
    T = rng.uniform(0.4, 1.6, B).astype(np.float32)
    m = rng.uniform(0.004, 0.4, B).astype(np.float32)
    M = (np.sign(rng.normal(size=B)) * 2.0 ** rng.uniform(2, 16, B)).astype(np.float32)
    for b in range(B):
        limit = float(M[b]) + float(T[b]) * np.log(float(m[b]))
        above = np.float32(limit)
        if float(above) < limit:
            above = np.nextafter(above, np.float32(np.inf))
        first, second, third = np.argsort(-g[b])[:3]
        x[b, first], x[b, second] = np.nextafter(above, np.float32(-np.inf)), above
        x[b, np.argsort(g[b])[0]] = M[b]                  # (the worst noise, so that its key is not the best)
    z = (x.astype(np.float64) - M[:, None]) / T[:, None]
    gap = np.abs(z - np.log(m.astype(np.float64))[:, None])
    # decided by more than the limit's own precision
    clear = gap.min(1) > 2.0 ** -22 * np.abs(np.log(m.astype(np.float64)))
    return x, T, m, clear


def test_rows_at_the_min_p_limit_are_decided():
    x, T, m, clear = cut_rows(400, 41)
    assert clear.mean() > 0.7
    ids, _ = fl.sample(x, T, np.zeros(400), np.ones(400), m, 41)
    g = -np.log(sm.exponential_noise(41, 0, range(400), 1024))
    assert (ids == np.argsort(-g, axis=1)[:, 1]).mean() > 0.9      # mostly the token at the limit, not the one below it


@pytest.mark.gpu
@pytest.mark.parametrize("B", [8, 40, 400])
def test_min_p_cuts_where_its_limit_is(pkv, B):
    """The limit is compared in the logits' own differences from the largest: large logits do not round it."""
    x, T, m, clear = cut_rows(B, 41)
    ref, margin = fl.sample(x, T, np.zeros(B), np.ones(B), m, 41)
    assert (margin[clear] > 1e-9).all()
    f = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    for k in (None, torch.full((B,), 3, dtype=torch.int32).cuda()):
        got = pkv.pkv_sample_filtered(f(x), f(T), k, None, f(m), 41).cpu().numpy()
        assert np.array_equal(got[clear], ref[clear]), (np.nonzero(clear & (got != ref))[0])
    expect_no_device_error(pkv)
