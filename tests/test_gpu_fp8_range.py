"""Decode over an 8-bit cache where few keys outweigh many, and where values are of any size the format holds.

Tolerance.  A key's weight times its value's scale is rounded to f16 relative to W, the largest such product
its warp has seen: to 2^-11 of itself, and to no less than 2^-38 of W (f16's smallest step is 2^-24, half of
it 2^-25, and the largest product is held at 2^13 or above).  With the codes c_j, that is 2^-11 A + 2^-38 W sum |c_j|
beside 2^-13 A for the scores and sums and 2^-8 of the output for its rounding to bf16, A = sum p_j |v_j|."""
import numpy as np
import pytest
import torch

from oracle import fp8_cache as fc
from pkv_testutil import expect_no_device_error

pytestmark = pytest.mark.gpu
D = 128
LN2 = 0.6931471805599453


def decode(pkv, score, v, ev, batch, hq=16, hkv=8):
    """`batch` equal sequences whose keys have these log2 scores (e4m3 numbers; element 0 of K), codes' values v [n, D]
    and scale exponents ev; returns the outputs and, in 64 bits, the result, A and the bound's W sum |c|."""
    n, bs = len(score), 256
    nb = -(-n // bs)
    score, v, ev = np.asarray(score, np.float64), np.asarray(v, np.float64), np.asarray(ev)
    k = np.zeros((nb * bs, hkv, D), np.uint8)
    k[:n, :, 0] = fc.round_e4m3(score)[:, None]
    assert np.array_equal(fc.E4M3[k[:n, 0, 0]], score)
    codes = np.full((nb * bs, hkv, D), 0x7f, np.uint8)
    codes[:n] = fc.round_e4m3(v)[:, None]
    assert np.array_equal(fc.E4M3[codes[:n, 0]], v)
    vs = np.full((nb * bs, hkv), 255, np.uint8)
    vs[:n] = (ev + 127)[:, None]
    q = torch.zeros(batch, hq, D, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).cuda().view(dt)  # noqa: E731
    out = pkv.pkv_decode_fp8(q.cuda(), t(k.reshape(nb, bs, hkv, D), torch.float8_e4m3fn), t(codes.reshape(nb, bs, hkv, D), torch.float8_e4m3fn),
                             t(np.full((nb, hkv, bs), 127, np.uint8), torch.float8_e8m0fnu),
                             t(vs.reshape(nb, bs, hkv).transpose(0, 2, 1), torch.float8_e8m0fnu),
                             torch.arange(nb, dtype=torch.int32).repeat(batch, 1).cuda(), torch.full((batch,), n, dtype=torch.int32).cuda(), n, LN2)
    w = 2.0 ** (score - score.max())
    w /= w.sum()
    x = (w * 2.0 ** ev)[:, None] * v
    expect_no_device_error(pkv)
    return out.double().cpu().numpy(), x.sum(0), np.abs(x).sum(0), (w * 2.0 ** ev).max() * np.abs(v).sum(0)


def within(got, ref, A, small):
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * A + 2.0 ** -38 * small
    err = np.abs(got - ref)
    assert np.isfinite(got).all() and np.all(err <= tol), (float(err.max()), float((err / np.where(tol == 0, 1e-300, tol)).max()))


@pytest.mark.parametrize("first,ev", [(14, 0), (18, 0), (20, 0), (20, 6), (24, 6), (28, 2)])
def test_many_light_keys_behind_a_heavy_one(pkv, first, ev):
    """The heavy key holds 0 in half of the channels, which the thousands of light ones make alone."""
    n, rng = 4000, np.random.default_rng(first + ev)
    score = np.where(np.arange(n) == 0, first, rng.choice([0.0, -0.5, -1.0, 0.25], n))
    v = fc.E4M3[fc.round_e4m3(rng.uniform(1, 400, (n, D)))]
    v[0, ::2] = 0
    got, ref, A, small = decode(pkv, score, v, np.where(np.arange(n) == 0, ev, 0), batch=200)
    # (light keys make the empty channels to a part in two hundred of themselves or better)
    assert np.all(2.0 ** -38 * small[::2] <= 0.005 * ref[::2])
    within(got, ref, A, small)


def test_heavy_keys_late_and_in_between(pkv):
    """The reference moves in the middle of a run, by a little and by much."""
    n, rng = 2000, np.random.default_rng(3)
    score = np.where(rng.random(n) < 0.01, rng.choice([2.0, 5.0, 9.0, 13.0, 15.0], n), rng.choice([0.0, -4.0, -11.0], n))
    score[1990] = 26.0
    ev = rng.integers(-6, 7, n)
    v = fc.E4M3[fc.round_e4m3(rng.normal(size=(n, D)) * 60)]
    v[:, 1::4] *= (score < 1)[:, None]
    for batch in (1, 200):
        within(*decode(pkv, score, v, ev, batch))


@pytest.mark.parametrize("exponent", [-126, -110, -60, 0, 60, 110, 118])
def test_values_of_every_size(pkv, exponent):
    """V of one size throughout, from the smallest scales to bf16's largest numbers, with scores that rise by 60 octaves."""
    n, rng = 300, np.random.default_rng(7)
    score = np.where(np.arange(n) < 32, 0.0, np.where(np.arange(n) < 250, 60.0, 56.0))
    v = fc.E4M3[fc.round_e4m3(rng.choice([-1, 1], (n, D)) * rng.uniform(64, 400, (n, D)))]
    for batch in (1, 160):
        within(*decode(pkv, score, v, np.full(n, exponent), batch))
