"""A key that a node does not see has no effect on its row, and neither have the rows beside it: the same bits, whatever
the keys of others hold and however a call's bounds are stated."""
import numpy as np
import pytest
import torch

from pkv_testutil import expect_no_device_error
from test_gpu_tree import Trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("nodes,context", [(4, 32), (4, 40), (8, 100), (30, 64), (30, 130), (100, 64)])
def test_large_keys_that_others_do_not_see(pkv, nodes, context, fp8):
    """A node that only it sees holds a K along its own query, large enough to move its row's reference: in every other row
    (of which some meet their largest score among the nodes, a little above the context's) nothing changes."""
    hidden = nodes // 2
    for seed in range(6):
        sees = np.tril(np.ones((nodes, nodes), bool))
        sees[:, hidden] = False
        sees[hidden, hidden] = True
        b = Trees([nodes], [context + nodes], 4, 2, seed=seed, masks=[sees], fp8=fp8)
        clean = b.gpu(pkv)
        b.check(clean)
        blk, off = b.at(0, context + hidden)
        along = torch.sign(b.q[hidden, ::2].float())                       # a query head of each KV head
        if fp8:
            b.kc[blk, off] = np.where(along.numpy() < 0, 0xfe, 0x7e)       # -448 or 448
            b.ks[blk, :, off] = 127
        b.k[blk, off] = (448 * along).bfloat16()
        out = b.gpu(pkv)
        expect_no_device_error(pkv)
        b.check(out)
        others = [i for i in range(nodes) if i != hidden]
        assert torch.equal(out[others], clean[others]), seed


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("nodes", [4, 30])
def test_any_bound_on_the_lengths(pkv, nodes, fp8):
    """The loosest bound there is, with so many sequences that their product passes 2^31 tiles: the same bits."""
    rng = np.random.default_rng(nodes)
    lens = nodes + rng.integers(0, 700, 130)
    b = Trees([nodes] * 130, lens, 4, 2, seed=nodes, fp8=fp8)
    tight = b.gpu(pkv)
    assert torch.equal(tight, b.gpu(pkv, max_len=2 ** 31 - 1))
    expect_no_device_error(pkv)
    b.check(tight, range(0, 130, 17))


@pytest.mark.parametrize("scale", [128 ** -0.5, 1e-9, 1e-30, 1e-44])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("nodes", [4, 40, 140])
def test_small_queries_and_scales(pkv, nodes, fp8, scale):
    """Scores that are all next to 0 weigh evenly what a row sees, and a row that sees nothing is zero: with queries of
    zero, of the smallest numbers and of none at all."""
    rng = np.random.default_rng(nodes)
    sees = rng.random((nodes, nodes)) < 0.4
    sees[np.arange(nodes), np.arange(nodes)] = True
    sees[[0, 3]] = False
    for context in (0, 200):
        b = Trees([nodes], [nodes + context], 4, 2, seed=nodes, masks=[sees], fp8=fp8)
        b.scale = scale
        b.q[::2] = 0.0
        b.q[1::2] *= 2.0 ** -125
        b.check(b.gpu(pkv))
    b = Trees([nodes], [nodes], 4, 2, seed=nodes, masks=[sees], fp8=fp8)
    b.scale = scale
    clean = b.gpu(pkv)
    b.q[0], b.q[3] = float("nan"), float("inf")        # they see nothing, themselves included
    out = b.gpu(pkv)
    assert not out[[0, 3]].any() and torch.equal(out, clean)
    expect_no_device_error(pkv)
