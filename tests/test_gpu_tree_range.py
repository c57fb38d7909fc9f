"""Attention of trees whose values are of any size their type holds: finite values give finite results.

Tolerance.  With A = sum p_j |v_j|: weights rounded to bf16 (2^-8 A), scores and sums in fp32 (2^-13 A), the output's own
rounding (2^-8 |ref|).  A row's weights sum to 2^-18 or more, so that sums in fp32, whose smallest step is 2^-149, are off
by 2^-131 of the result's unit a step at most, and less than 2^-128 in all where few steps count."""
import numpy as np
import pytest
import torch

from oracle import fp8_cache as fc
from pkv_testutil import expect_no_device_error

pytestmark = pytest.mark.gpu
D = 128
LN2 = 0.6931471805599453


def attend(pkv, score, v, ev, nodes, batch, fp8, hq=2, hkv=2):
    """`batch` equal sequences whose keys have these log2 scores (element 0 of K) and the values v [n, D] 2^ev; every node
    sees every key.  Returns the outputs and, in 64 bits, the result and A."""
    n, bs = len(score), 256
    nb = -(-n // bs)
    score, v, ev = np.asarray(score, np.float64), np.asarray(v, np.float64), np.asarray(ev)
    q = torch.zeros(batch * nodes, hq, D, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    words = -(-nodes // 64)
    rest = (torch.arange(nb, dtype=torch.int32).repeat(batch, 1).cuda(), torch.full((batch,), n, dtype=torch.int32).cuda(),
            (torch.arange(batch + 1, dtype=torch.int32) * nodes).cuda(), torch.full((batch * nodes, words), -1, dtype=torch.int64).cuda(),
            nodes, n, LN2)
    if fp8:
        k = np.zeros((nb * bs, hkv, D), np.uint8)
        k[:n, :, 0] = fc.round_e4m3(score)[:, None]
        assert np.array_equal(fc.E4M3[k[:n, 0, 0]], score)
        codes = np.full((nb * bs, hkv, D), 0x7f, np.uint8)
        codes[:n] = fc.round_e4m3(v)[:, None]
        assert np.array_equal(fc.E4M3[codes[:n, 0]], v)
        vs = np.full((nb * bs, hkv), 255, np.uint8)
        vs[:n] = (ev + 127)[:, None]
        t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).cuda().view(dt)  # noqa: E731
        out = pkv.pkv_tree_decode_fp8(q.cuda(), t(k.reshape(nb, bs, hkv, D), torch.float8_e4m3fn), t(codes.reshape(nb, bs, hkv, D), torch.float8_e4m3fn),
                                      t(np.full((nb, hkv, bs), 127, np.uint8), torch.float8_e8m0fnu),
                                      t(vs.reshape(nb, bs, hkv).transpose(0, 2, 1), torch.float8_e8m0fnu), *rest)
    else:
        k = torch.full((nb * bs, hkv, D), float("nan"), dtype=torch.bfloat16)
        values = k.clone()
        k[:n] = 0
        k[:n, :, 0] = torch.from_numpy(score).bfloat16()[:, None]
        values[:n] = torch.from_numpy(np.ldexp(v, ev[:, None])).bfloat16()[:, None]
        assert np.array_equal(k[:n, 0, 0].double().numpy(), score) and np.array_equal(values[:n, 0].double().numpy(), np.ldexp(v, ev[:, None]))
        out = pkv.pkv_tree_decode(q.cuda(), k.view(nb, bs, hkv, D).cuda(), values.view(nb, bs, hkv, D).cuda(), *rest)
    expect_no_device_error(pkv)
    w = 2.0 ** (score - score.max())
    x = np.ldexp((w / w.sum())[:, None] * v, ev[:, None])
    return out.double().cpu().numpy(), x.sum(0), np.abs(x).sum(0)


def within(got, ref, A):
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -13) * A + 2.0 ** -128
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), np.argwhere(~np.isfinite(got))[:4]
    assert np.all(err <= tol), (float(err.max()), float((err / tol).max()))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("nodes", [8, 17, 64])
@pytest.mark.parametrize("exponent", [-126, -110, -60, 0, 60, 110, 118])
def test_values_of_every_size(pkv, exponent, nodes, fp8):
    """V of one size throughout, from the smallest scales to bf16's largest numbers, with scores that rise by 60 octaves."""
    n, rng = 300, np.random.default_rng(7)
    score = np.where(np.arange(n) < 32, 0.0, np.where(np.arange(n) < 250, 60.0, 56.0))
    v = fc.E4M3[fc.round_e4m3(rng.choice([-1, 1], (n, D)) * rng.uniform(64, 400, (n, D)))]
    for batch in (1, 90):
        within(*attend(pkv, score, v, np.full(n, exponent), nodes, batch, fp8))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("nodes", [8, 17, 64, 130])
@pytest.mark.parametrize("n,rise", [(130, 0), (2000, 0), (2000, 7.5), (40000, 0), (40000, 7.5), (40000, 20)])
def test_sums_of_the_largest_values(pkv, n, rise, nodes, fp8):
    """Keys of equal weight, or of weights that grow along the sequence, all with values of 2^126 and some of either sign."""
    score = fc.E4M3[fc.round_e4m3(np.linspace(0, rise, n))]
    v = np.full((n, D), 256.0)
    v[:, 1::2] = np.where(np.random.default_rng(n).random((n, D // 2)) < 0.3, -256.0, 256.0)
    for batch in (1, 40) if n < 40000 else (1,):
        within(*attend(pkv, score, v, np.full(n, 118), nodes, batch, fp8))


def test_two_keys_of_the_largest_power(pkv):
    """2^127 twice, at equal weight."""
    for nodes in (1, 20):
        got, ref, A = attend(pkv, np.zeros(nodes + 1), np.full((nodes + 1, D), 128.0), np.full(nodes + 1, 120), nodes, 1, False)
        assert np.all(got == 2.0 ** 127)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("nodes", [8, 40])
def test_light_keys_with_large_values(pkv, nodes, fp8):
    """Keys far below the heaviest make the channels in which that one holds 0."""
    n, rng = 3000, np.random.default_rng(5)
    score = np.where(np.arange(n) == 40, 28.0, rng.choice([0.0, -0.5, -1.0, 0.25], n))
    v = fc.E4M3[fc.round_e4m3(rng.uniform(1, 400, (n, D)))]
    v[40, ::2] = 0
    for ev in (0, 100):
        within(*attend(pkv, score, v, np.where(np.arange(n) == 40, 0, ev), nodes, 1, fp8))
