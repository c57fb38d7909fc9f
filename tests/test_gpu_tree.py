"""Decoding along a tree of drafted tokens on the GPU, against float64.

Tolerances.  With A = sum_j p_j |v_j| per output element: a key's weight is rounded to bf16
(2^-8 A), scores and sums are fp32 (a score error of 2^-13 would be 1000 roundings of a score near 1;
2^-13 A), the output is rounded once to bf16 (2^-8 |ref|).  The 8-bit attention multiplies the codes
themselves by two e4m3 parts of each query, off by 2^-18 of the row's largest at most.  Paths, moved rows and copied blocks are exact."""
import numpy as np
import pytest
import torch

from oracle import fp8_cache as fc
from oracle import tree as tr
from pkv_testutil import expect_no_device_error

pytestmark = pytest.mark.gpu
D = 128
NAN = float("nan")


def random_tree(n, rng, reach=6):
    """Ancestors (self included) of a random tree, boolean [n, n]."""
    sees = np.eye(n, dtype=bool)
    for i in range(1, n):
        sees[i] |= sees[max(0, i - 1 - int(rng.integers(0, reach)))]
    return sees


class Trees:
    """A batch of sequences with trees of drafts, on a paged cache that holds NaN wherever no sequence has a row."""

    def __init__(self, nodes, lens, hq, hkv, block=256, seed=0, fp8=False, masks=None, words=None, spare_rows=0, width=0):
        rng = np.random.default_rng(seed)
        self.n, self.len, self.hq, self.hkv, self.block, self.fp8 = list(nodes), list(lens), hq, hkv, block, fp8
        need = [-(-x // block) for x in lens]
        self.nb = sum(need) + 2
        perm = rng.permutation(self.nb)
        self.tables = np.full((len(lens), max([1, width] + need)), -1, np.int32)
        at = 0
        for s, m in enumerate(need):
            self.tables[s, :m] = perm[at:at + m]
            at += m
        self.most = max([1] + self.n)
        self.words = words or -(-self.most // 64)
        self.cu = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        total = int(self.cu[-1]) + spare_rows
        self.sees = [random_tree(x, rng) for x in self.n] if masks is None else masks
        self.mask = np.zeros((total, self.words), np.uint64)
        for s, x in enumerate(self.n):
            if x:
                self.mask[self.cu[s]:self.cu[s] + x] = tr.words_of(self.sees[s], self.words)
        g = torch.Generator().manual_seed(seed)
        self.q = torch.randn(total, hq, D, generator=g).bfloat16()
        self.k = torch.full((self.nb, block, hkv, D), NAN, dtype=torch.bfloat16)
        self.v = self.k.clone()
        if fp8:
            self.kc, self.vc = (np.full((self.nb, block, hkv, D), 0x7f, np.uint8) for _ in "kv")
            self.ks, self.vs = (np.full((self.nb, hkv, block), 255, np.uint8) for _ in "kv")
        for s, length in enumerate(lens):
            for j in range(need[s]):
                m, b = min(block, length - j * block), self.tables[s, j]
                if fp8:
                    for codes, scales in ((self.kc, self.ks), (self.vc, self.vs)):
                        codes[b, :m] = rng.integers(0, 127, (m, hkv, D)) | (rng.integers(0, 2, (m, hkv, D)) << 7)
                        scales[b, :, :m] = 119 + rng.integers(-2, 3, (hkv, m))
                else:
                    self.k[b, :m] = torch.randn(m, hkv, D, generator=g).bfloat16()
                    self.v[b, :m] = torch.randn(m, hkv, D, generator=g).bfloat16()
        if fp8:
            with np.errstate(invalid="ignore"):
                self.k = torch.from_numpy(fc.read_pool(self.kc, self.ks)).bfloat16()
                self.v = torch.from_numpy(fc.read_pool(self.vc, self.vs)).bfloat16()
        self.scale = D ** -0.5

    def at(self, s, pos):
        return int(self.tables[s, pos // self.block]), pos % self.block

    def gpu(self, lib, as_bf16=False, out=None, workspace=None, stream=None, max_len=None):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        lens = torch.tensor(self.len, dtype=torch.int32).cuda()
        mask = dev(self.mask.view(np.int64))
        rest = (dev(self.tables), lens, dev(self.cu), mask, self.most, max_len or max([1] + self.len), self.scale)
        kw = dict(out=out, workspace=workspace, stream=stream)
        if self.fp8 and not as_bf16:
            pools = (dev(self.kc).view(torch.float8_e4m3fn), dev(self.vc).view(torch.float8_e4m3fn),
                     dev(self.ks).view(torch.float8_e8m0fnu), dev(self.vs).view(torch.float8_e8m0fnu))
            return lib.pkv_tree_decode_fp8(self.q.cuda(), *pools, *rest, **kw)
        return lib.pkv_tree_decode(self.q.cuda(), self.k.cuda(), self.v.cuda(), *rest, **kw)

    def rows(self, pool, s):
        b = self.tables[s, :-(-self.len[s] // self.block)].astype(np.int64)
        return pool[b].reshape(-1, self.hkv, D)[:self.len[s]].double().numpy()

    def check(self, out, seqs=None):
        got = out.double().cpu().numpy()
        for s in range(len(self.n)) if seqs is None else seqs:
            if not self.n[s]:
                continue
            lo, hi = self.cu[s], self.cu[s + 1]
            ref, A = tr.attention(self.q[lo:hi].double().numpy(), self.rows(self.k, s), self.rows(self.v, s), self.sees[s], self.scale)
            with np.errstate(invalid="ignore"):
                off = np.abs(got[lo:hi] - ref) - (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -13) * A + 1e-30)
            fine = np.isfinite(ref)
            assert np.array_equal(np.isfinite(got[lo:hi]), fine), (s, np.argwhere(np.isfinite(got[lo:hi]) != fine)[:4])
            assert np.all(off[fine] <= 0), (s, float(off[fine].max()), np.argwhere(fine & ~(off <= 0))[:4])


BATCHES = {
    "one node, one key": ([1], [1]),
    "one node": ([1], [70]),
    "tile borders": ([3, 5, 64, 1, 7], [64, 128, 128, 65, 257]),
    "no context": ([5, 64, 33], [5, 64, 33]),
    "ragged": ([0, 9, 31, 1, 0, 64, 17], [0, 100, 31, 513, 40, 600, 255]),
    "long trees": ([65, 200, 256, 129], [300, 200, 700, 1025]),
    "split over its length": ([13], [9001]),
    "two long": ([64, 40], [5000, 7001]),
}
HEADS = [(16, 8), (4, 4), (8, 1), (8, 2)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("name", BATCHES)
def test_attention(pkv, name, hq, hkv, fp8):
    nodes, lens = BATCHES[name]
    b = Trees(nodes, lens, hq, hkv, block=512 if hkv == 4 else 256, seed=len(name) + hq, fp8=fp8)
    out = b.gpu(pkv)
    expect_no_device_error(pkv)
    b.check(out)


SMALL = {
    "single nodes": ([1, 1, 1, 1, 1], [1, 31, 32, 33, 700]),
    "chunk borders": ([2, 4, 3, 1, 4], [32, 64, 63, 65, 257]),
    "no context": ([4, 1, 2], [4, 1, 2]),
    "ragged": ([0, 3, 4, 0, 0, 1, 2], [5, 100, 36, 0, 40, 600, 255]),
    "split over its length": ([3], [9001]),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 4), (6, 3)])
@pytest.mark.parametrize("name", SMALL)
def test_small_trees(pkv, name, hq, hkv, fp8):
    """Up to 4 nodes: 4 to 16 rows."""
    nodes, lens = SMALL[name]
    b = Trees(nodes, lens, hq, hkv, seed=hq + hkv, fp8=fp8)
    out = b.gpu(pkv)
    expect_no_device_error(pkv)
    b.check(out)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("most", [4, 8, 9, 16, 17, 32, 33])
def test_results_do_not_depend_on_bounds(pkv, most, fp8):
    """Loose bounds on the lengths give the same bits; a tree's rows do not depend on the rest of the batch's sizes."""
    b = Trees([most, 2, most], [800, 2600, most + 1], 2, 2, seed=most, fp8=fp8)
    tight = b.gpu(pkv)
    assert torch.equal(tight, b.gpu(pkv, max_len=70000))
    b.check(tight)


@pytest.mark.parametrize("power", [-60, 0, 60])
@pytest.mark.parametrize("nodes", [4, 12])
def test_value_scales_far_apart_8_bits(pkv, nodes, power):
    """Scales of V that differ by 2^80 from key to key: the large ones' rows are right, whatever the order they come in."""
    b = Trees([nodes], [300], 2, 1, seed=3, fp8=True)
    rng = np.random.default_rng(4)
    owned = b.vs != 255
    b.vs[owned] = 127 + power // 2 + rng.integers(-40, 41, int(owned.sum()))
    b.v = torch.from_numpy(fc.read_pool(b.vc, b.vs)).bfloat16()
    b.check(b.gpu(pkv))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("nodes", [4, 12, 40])
@pytest.mark.parametrize("bad", [float("inf"), NAN])
def test_bad_queries_stay_in_their_rows(pkv, bad, nodes, fp8):
    b = Trees([nodes, 3], [500, 90], 4, 2, seed=6, fp8=fp8)
    clean = b.gpu(pkv)
    b.q[2, 1, 5] = bad
    b.q[nodes + 1, 3] = bad
    out = b.gpu(pkv)
    hit = torch.zeros(nodes + 3, 4, dtype=torch.bool)
    hit[2, 1] = hit[nodes + 1, 3] = True
    assert torch.isnan(out[hit.cuda()]).all()
    assert torch.equal(out[~hit.cuda()], clean[~hit.cuda()])


def test_keys_first_seen_late(pkv):
    """Rows that see nothing in the first tiles and then only keys with very low scores."""
    n = 140
    sees = np.zeros((n, n), bool)
    sees[:, 100:] = np.random.default_rng(2).random((n, 40)) < 0.5
    sees[7] = False
    b = Trees([n], [n], 2, 1, seed=5, masks=[sees])
    for i in range(100, n):
        blk, off = b.at(0, i)
        b.k[blk, off, 0] = -4 * b.q[7, 0]              # far below 0 for many rows
    b.q[:] = b.q[7:8, :1]
    out = b.gpu(pkv)
    b.check(out)
    assert not out[7].any()
    c = Trees([4], [4], 2, 1, seed=5, masks=[np.array([[0, 0, 0, 1]] * 3 + [[0, 0, 0, 0]], bool)], fp8=True)
    c.check(c.gpu(pkv))


def test_codes_that_read_as_nan_8_bits(pkv):
    """NaN codes of K and of V reach the rows that see them, on the kernels for few rows and for many."""
    for nodes in (4, 30):
        sees = np.tril(np.ones((nodes, nodes), bool))
        sees[:, 1] = False
        sees[[1, 3], 1] = True
        b = Trees([nodes], [200], 4, 2, seed=8, masks=[sees], fp8=True)
        clean = b.gpu(pkv)
        blk, off = b.at(0, 200 - nodes + 1)
        seen = torch.tensor([i in (1, 3) for i in range(nodes)]).cuda()
        kept = b.vc[blk, off].copy()
        b.vc[blk, off, :, 100] = 0xff
        out = b.gpu(pkv)
        others = torch.arange(D).cuda() != 100
        assert torch.isnan(out[seen][..., 100]).all() and torch.equal(out[~seen], clean[~seen])
        assert torch.equal(out[..., others], clean[..., others])
        b.vc[blk, off] = kept
        b.kc[blk, off, 0, 9] = 0x7f                    # KV head 0: query heads 0 and 1
        out = b.gpu(pkv)
        assert torch.isnan(out[seen][:, :2]).all() and torch.equal(out[~seen], clean[~seen]) and torch.equal(out[:, 2:], clean[:, 2:])
        b.ks[blk, :, off] = 255                        # both heads' rows of K
        out = b.gpu(pkv)
        assert torch.isnan(out[seen]).all() and torch.equal(out[~seen], clean[~seen])


def test_two_calls_at_once(pkv):
    """Two streams, a workspace each."""
    a, b = Trees([64, 40], [9000, 3000], 16, 8, seed=1), Trees([4, 3], [20000, 7000], 16, 8, seed=2, fp8=True)
    wa, wb = a.gpu(pkv), b.gpu(pkv)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        oa, ob = a.gpu(pkv, stream=sa), b.gpu(pkv, stream=sb)
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_wrong_arguments(pkv):
    b = Trees([4], [40], 4, 2, seed=1)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    q, k, v = b.q.cuda(), b.k.cuda(), b.v.cuda()
    tab, lens, cu, mask = dev(b.tables), torch.tensor(b.len, dtype=torch.int32).cuda(), dev(b.cu), dev(b.mask.view(np.int64))
    call = lambda q=q, k=k, v=v, tab=tab, lens=lens, cu=cu, mask=mask, nodes=4, **kw: pkv.pkv_tree_decode(  # noqa: E731
        q, k, v, tab, lens, cu, mask, nodes, 40, 0.1, **kw)
    call()
    for bad in ({"q": q.float()}, {"lens": lens.long()}, {"mask": mask.int()}):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in ({"q": q[:3]}, {"cu": cu[:1]}, {"mask": mask[:2]}, {"tab": tab.repeat(2, 1)}, {"v": v[:1]}, {"q": q.transpose(0, 1)},
                {"out": torch.empty(5, 4, D, dtype=torch.bfloat16).cuda()}, {"mask": mask.cpu()}, {"q": q[..., :64].contiguous()}):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in ({"nodes": 65}, {"workspace": torch.empty(256, dtype=torch.uint8).cuda()}, {"out": q}):
        with pytest.raises(pkv.PkvError):
            call(**bad)
    expect_no_device_error(pkv)
    pool = lambda: torch.zeros(2, 256, 2, D, dtype=torch.bfloat16).cuda()  # noqa: E731
    x = pool()
    for k_list, v_list in (([x], [x]), ([x, x], [pool(), pool()]), ([x], [x[:1]]), ([x], [pool(), pool()]), ([pool(), pool()[:1]], [pool(), pool()])):
        with pytest.raises(ValueError):
            pkv.KvPools(k_list, v_list)
    with pytest.raises(TypeError):
        pkv.KvPools([x.half()], [pool()])
    pools = pkv.KvPools([x], [pool()])
    with pytest.raises(ValueError):
        pkv.pkv_copy_blocks(pools, torch.zeros(2, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda())
    with pytest.raises(ValueError):
        pkv.pkv_copy_blocks(pools, torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
def test_many_short_sequences(pkv, fp8):
    """More sequences than a CTA has threads, some of them empty; a run crosses many of them."""
    rng = np.random.default_rng(5)
    nodes = rng.integers(0, 5, 1500)
    lens = nodes + rng.integers(0, 40, 1500)
    b = Trees(nodes, lens, 2, 1, seed=6, fp8=fp8)
    out = b.gpu(pkv)
    expect_no_device_error(pkv)
    b.check(out, range(0, 1500, 7))


def test_the_largest_batch(pkv):
    b = Trees([1] * 4096, [1 + i % 3 for i in range(4096)], 1, 1, seed=2)
    b.check(b.gpu(pkv), range(0, 4096, 97))
    c = Trees([1] * 4097, [1] * 4097, 1, 1, seed=2)
    with pytest.raises(pkv.PkvError, match="UNSUPPORTED"):
        c.gpu(pkv)
    expect_no_device_error(pkv)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
def test_any_mask(pkv, fp8):
    """Masks that are no tree: random bits, nothing at all, everything, and bits behind the last node."""
    rng = np.random.default_rng(9)
    nodes, lens = [70, 40, 33, 64], [70, 300, 33, 64 + 19]
    masks = [rng.random((n, n)) < 0.3 for n in nodes]
    masks[0][5] = masks[0][69] = False                 # no context: these rows see nothing
    masks[2][:] = False
    masks[3][:] = True
    b = Trees(nodes, lens, 8, 2, seed=10, fp8=fp8, masks=masks)
    b.mask[b.cu[1]:b.cu[2], 0] |= ~np.uint64((1 << 40) - 1)
    b.mask[b.cu[1]:b.cu[2], 1] = ~np.uint64(0)
    out = b.gpu(pkv)
    expect_no_device_error(pkv)
    b.check(out)
    assert not out[b.cu[2]:b.cu[3]].any() and not out[5].any() and not out[69].any()


def test_more_words_than_needed(pkv):
    a = Trees([20, 7], [90, 300], 8, 2, seed=3)
    b = Trees([20, 7], [90, 300], 8, 2, seed=3, words=6)
    assert torch.equal(a.gpu(pkv), b.gpu(pkv))


def test_a_chain_is_causal(pkv):
    """A tree without branches: the causal attention of a chunk behind its prefix."""
    nodes, lens = [40, 17], [500, 1000]
    b = Trees(nodes, lens, 16, 8, seed=4, masks=[np.tril(np.ones((n, n), bool)) for n in nodes])
    out = b.gpu(pkv)
    cu_k = torch.tensor([0, 500, 1500], dtype=torch.int32).cuda()
    ref = pkv.pkv_prefill_varlen(b.q.cuda(), b.k.cuda(), b.v.cuda(), torch.from_numpy(b.cu).cuda(), cu_k,
                                 torch.from_numpy(b.tables).cuda(), 40, 1000, b.scale)
    b.check(out)
    b.check(ref)


@pytest.mark.parametrize("length", [150, 5000])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), NAN])
def test_unseen_rows_have_no_effect(pkv, bad, length):
    """Nodes that only they themselves see hold infinities or NaN in K and V: the others' rows are as without them."""
    n = 30
    sees = np.tril(np.random.default_rng(1).random((n, n)) < 0.5) | np.eye(n, dtype=bool)
    hidden = [3, 11, 29]
    sees[:, hidden] = False
    sees[hidden, hidden] = True
    b = Trees([n], [length], 8, 2, seed=8, masks=[sees])
    clean = b.gpu(pkv)
    for i in hidden:
        blk, off = b.at(0, length - n + i)
        b.v[blk, off, :, ::3] = bad
        if i != 11:
            b.k[blk, off] = bad
    out = b.gpu(pkv)
    expect_no_device_error(pkv)
    others = [i for i in range(n) if i not in hidden]
    assert torch.equal(out[others], clean[others])
    # node 11 sees itself: its K is fine, every third value is not
    assert not torch.isfinite(out[11, :, ::3]).any()
    keep = torch.ones(D, dtype=torch.bool)
    keep[::3] = False
    assert torch.equal(out[11][:, keep.cuda()], clean[11][:, keep.cuda()])


def test_rows_that_cannot_be_read_8_bits(pkv):
    """A row with scale 255 reads as NaN: it reaches the nodes that see it and no other."""
    n, length = 20, 400
    sees = np.tril(np.ones((n, n), bool))
    sees[:, 4] = False
    sees[[4, 9], 4] = True
    b = Trees([n], [length], 4, 2, seed=8, masks=[sees], fp8=True)
    clean = b.gpu(pkv)
    blk, off = b.at(0, length - n + 4)
    scales = b.vs[blk, :, off].copy()
    b.vs[blk, :, off] = 255
    out = b.gpu(pkv)
    seen = torch.tensor([i in (4, 9) for i in range(n)]).cuda()
    assert torch.isnan(out[seen]).all() and torch.equal(out[~seen], clean[~seen])
    b.vc[blk, off, :, 7] = 0x7f                        # a NaN code beside a proper scale
    b.vs[blk, :, off] = scales
    out = b.gpu(pkv)
    assert torch.isnan(out[seen][..., 7]).all() and torch.equal(out[~seen], clean[~seen])
    keep = torch.arange(D).cuda() != 7
    assert torch.equal(out[..., keep], clean[..., keep])


def test_large_scores_and_values(pkv):
    b = Trees([25], [333], 8, 2, seed=12)
    b.q *= 30
    b.v *= 2.0 ** 100
    b.check(b.gpu(pkv))


@pytest.mark.parametrize("power", [-100, 0, 3, 12])
def test_large_and_small_queries_8_bits(pkv, power):
    """Scores of any size up to some hundreds: a query's two parts and the codes' products lose nothing that counts
    (2^-18 of the row's largest |q| in each of 128 products with |k| < 4 is below 2^-9 q_max / sqrt(128), on a
    score that such a row's own keys put near q_max sqrt(128))."""
    b = Trees([25, 64], [333, 2000], 8, 2, seed=12, fp8=True)
    b.q *= 2.0 ** power / 12
    b.ks[:] = np.where(b.ks == 255, 255, b.ks - 4)
    b.k = torch.from_numpy(fc.read_pool(b.kc, b.ks)).bfloat16()
    if power == -100:
        b.ks[:] = np.where(b.ks == 255, 255, b.ks + 100)
        b.k = torch.from_numpy(fc.read_pool(b.kc, b.ks)).bfloat16()
    b.check(b.gpu(pkv))


@pytest.mark.parametrize("down", [False, True], ids=["up", "down"])
@pytest.mark.parametrize("nodes", [3, 20, 70])
def test_scores_that_grow_along_the_keys_8_bits(pkv, nodes, down):
    """A row's reference moves again and again, in every part of a tile, and what has been weighed and summed moves with it.
    The queries are 1 or -1 and a key's elements are one code, so that scores (up to 170) are exact but for fp32 roundings."""
    b = Trees([nodes, 1], [900, 333], 4, 2, seed=61, fp8=True)
    b.q[:] = 1.0
    b.q[::3] = -1.0                                    # for these rows the scores fall
    for s, n in enumerate(b.len):
        for i in range(n):
            blk, off = b.at(s, i)
            code = min(126, 40 + 64 * (n - 1 - i if down else i) // n)
            b.kc[blk, off], b.ks[blk, :, off] = code, 127 - 2
    with np.errstate(invalid="ignore"):
        b.k = torch.from_numpy(fc.read_pool(b.kc, b.ks)).bfloat16()
    b.check(b.gpu(pkv))


def test_rows_left_alone(pkv):
    """Rows behind the last sequence, and sequences that break the bounds, stay as they were."""
    b = Trees([5, 9, 4], [40, 70, 30], 8, 2, seed=13, spare_rows=3)
    out = torch.full_like(b.q, 7.0).cuda()
    b.gpu(pkv, out=out)
    b.check(out)
    assert (out[18:] == 7.0).all()
    expect_no_device_error(pkv)
    for change in ("short", "long", "decreasing", "many"):
        c = Trees([5, 9, 4], [40, 70, 30], 8, 2, seed=13, spare_rows=3)
        kw = {}
        if change == "short":
            c.len[1] = 8                               # fewer keys than nodes
        elif change == "long":
            kw["max_len"] = 60
        elif change == "many":
            c.most = 8
        else:
            c.cu = np.array([0, 9, 5, 18], np.int32)
        out = torch.full_like(c.q, 7.0).cuda()
        c.gpu(pkv, out=out, **kw)
        code, info = pkv.pkv_get_device_error(clear=True)
        assert code == 3 and (info == 1 or change == "decreasing"), change
        if change != "decreasing":
            assert (out[5:14] == 7.0).all() and (out[18:] == 7.0).all()
            c.check(out, [0, 2])


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
def test_bad_block_ids_are_recorded(pkv, fp8):
    b = Trees([5, 9], [400, 700], 8, 2, seed=14, fp8=fp8)
    b.tables[1, 1] = b.nb + 5
    out = b.gpu(pkv)
    assert pkv.pkv_get_device_error(clear=True) == (1, 1)
    b.check(out, [0])
    b.tables[1, 1] = -1
    b.gpu(pkv)
    assert pkv.pkv_get_device_error(clear=True) == (1, 1)


def test_streams_workspaces_and_graphs(pkv):
    """The same bits every time: on another stream, from two captured graphs that share a workspace, replayed."""
    a, b = Trees([30, 12], [3000, 900], 16, 8, seed=15), Trees([64], [2500], 16, 8, seed=16, fp8=True)
    wa, wb = a.gpu(pkv), b.gpu(pkv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with_stream = a.gpu(pkv, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(with_stream, wa)
    ws = pkv.tree_decode_workspace(2, 64, 16, 8, D)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    qa, oa, qb, ob = a.q.cuda(), torch.zeros_like(a.q).cuda(), b.q.cuda(), torch.zeros_like(b.q).cuda()
    ka, va, ta, la, ca, ma = a.k.cuda(), a.v.cuda(), dev(a.tables), torch.tensor(a.len, dtype=torch.int32).cuda(), dev(a.cu), dev(a.mask.view(np.int64))
    pools = (dev(b.kc).view(torch.float8_e4m3fn), dev(b.vc).view(torch.float8_e4m3fn), dev(b.ks).view(torch.float8_e8m0fnu), dev(b.vs).view(torch.float8_e8m0fnu))
    tb, lb, cb, mb = dev(b.tables), torch.tensor(b.len, dtype=torch.int32).cuda(), dev(b.cu), dev(b.mask.view(np.int64))
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(ga):
        pkv.pkv_tree_decode(qa, ka, va, ta, la, ca, ma, 64, 4096, a.scale, out=oa, workspace=ws)
    with torch.cuda.graph(gb):
        pkv.pkv_tree_decode_fp8(qb, *pools, tb, lb, cb, mb, 64, 4096, b.scale, out=ob, workspace=ws)
    for _ in range(5):
        oa.zero_(), ob.zero_()
        ga.replay(), gb.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)
    la[0] = 2990                                       # the lengths are read when the graph runs
    ga.replay()
    torch.cuda.synchronize()
    a.len[0] = 2990
    assert torch.equal(oa, a.gpu(pkv))
    expect_no_device_error(pkv)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("nodes", [4, 30])
def test_graphs_of_any_shape(pkv, nodes, fp8):
    """Captured as a graph's first node, behind a memset, a copy and a join of two streams, and twice in a row on one workspace:
    a call starts beside the end of the kernel before it, and reads nothing before that has ended."""
    b = Trees([nodes, 2], [2000, 700], 8, 4, seed=31, fp8=fp8)
    want = b.gpu(pkv)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    q0, lens, cu, mask, tab = b.q.cuda(), torch.tensor(b.len, dtype=torch.int32).cuda(), dev(b.cu), dev(b.mask.view(np.int64)), dev(b.tables)
    if fp8:
        pools = (dev(b.kc).view(torch.float8_e4m3fn), dev(b.vc).view(torch.float8_e4m3fn), dev(b.ks).view(torch.float8_e8m0fnu), dev(b.vs).view(torch.float8_e8m0fnu))
        attend = pkv.pkv_tree_decode_fp8
    else:
        pools, attend = (b.k.cuda(), b.v.cuda()), pkv.pkv_tree_decode
    q, scratch, ws = torch.empty_like(q0), torch.empty(1 << 24, device="cuda"), pkv.tree_decode_workspace(2, nodes, 8, 4, D)
    outs = [torch.empty_like(q0) for _ in range(5)]
    call = lambda i: attend(q, *pools, tab, lens, cu, mask, nodes, 2000, b.scale, out=outs[i], workspace=ws)  # noqa: E731
    q.copy_(q0)
    other, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(0)
        q.zero_()
        scratch.zero_()
        q.copy_(q0)                                    # a copy node
        call(1)
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            q.zero_()
            scratch.add_(1.0)
            q.add_(q0)                                 # of the stream that is joined
        scratch2 = scratch.new_zeros(8)
        torch.cuda.current_stream().wait_stream(other)
        call(2)
        call(3)
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            call(4)                                    # the forked stream's first
        torch.cuda.current_stream().wait_stream(other)
        outs[0].add_(0.0)
        scratch2.zero_()
    for _ in range(3):
        for o in outs:
            o.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, want)
    expect_no_device_error(pkv)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
def test_blocks_far_into_a_pool(pkv, fp8):
    """Blocks more than 2^32 bytes (8 bits) or 2^31 elements (bf16) into their pools, for every call of a step."""
    hkv, block = 8, 256
    trees = [Trees([x, 1], [600, 40], 16, hkv, seed=41, fp8=fp8) for x in (4, 40)]
    nb = max(b.nb for b in trees)
    first = 2 ** 32 // (block * hkv * D * (1 if fp8 else 2)) + 1
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    byte = lambda *shape: torch.empty(*shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    if fp8:
        raw = [byte(first + nb, block, hkv, D) for _ in "kv"] + [byte(first + nb, hkv, block) for _ in "kv"]
        pools = [x.view(torch.float8_e4m3fn if i < 2 else torch.float8_e8m0fnu) for i, x in enumerate(raw)]
    else:
        raw = pools = [torch.empty(first + nb, block, hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    assert pools[0].numel() > 2 ** 31 and pools[0].numel() * pools[0].element_size() > 2 ** 32
    for b in trees:
        for x, h in zip(raw, (b.kc, b.vc, b.ks, b.vs) if fp8 else (b.k, b.v)):
            x[first:first + b.nb] = dev(h) if fp8 else h.cuda()
        tab = dev(np.where(b.tables < 0, -1, b.tables + first).astype(np.int32))
        lens, cu = torch.tensor(b.len, dtype=torch.int32).cuda(), dev(b.cu)
        attend = pkv.pkv_tree_decode_fp8 if fp8 else pkv.pkv_tree_decode
        out = attend(b.q.cuda(), *pools, tab, lens, cu, dev(b.mask.view(np.int64)), b.most, 600, b.scale)
        assert torch.equal(out, b.gpu(pkv))
        b.check(out)
        layers = pkv.KvPools(*[[x] for x in pools])
        n = b.n[0]
        pkv.pkv_tree_compact(layers, tab, lens, cu, dev(np.array([[0, n - 1], [0, -1]], np.int32)), dev(np.array([2, 1], np.int32)))
        spare = min(set(range(b.nb)) - set(b.tables[b.tables >= 0].tolist()))
        i32 = lambda x: torch.tensor([x], dtype=torch.int32).cuda()  # noqa: E731
        moved, to = b.at(0, 599), b.at(0, 600 - n + 1)
        pkv.pkv_copy_blocks(layers, i32(first + to[0]), i32(first + spare), i32(to[1] + 1))
        expect_no_device_error(pkv)
        for i, x in enumerate(raw):
            pick = (lambda at: x[at[0] + first, at[1]]) if i < 2 else (lambda at: x[at[0] + first, :, at[1]])  # noqa: B023
            assert torch.equal(pick(to).view(torch.uint8), pick(moved).view(torch.uint8))
            assert torch.equal(pick((spare, to[1])).view(torch.uint8), pick(moved).view(torch.uint8))


@pytest.mark.parametrize("nodes", [4, 140])
def test_queries_of_zero_8_bits(pkv, nodes):
    """Zero rows weigh what they see evenly, behind tiles of which they see nothing."""
    sees = np.zeros((nodes, nodes), bool)
    sees[:, -2:] = True
    sees[0] = False
    b = Trees([nodes], [nodes], 2, 1, seed=51, masks=[sees], fp8=True)
    b.q.zero_()
    out = b.gpu(pkv)
    b.check(out)
    assert not out[0].any()


def test_empty_calls(pkv):
    b = Trees([0, 0], [0, 30], 8, 2, seed=1, spare_rows=2)
    out = torch.full_like(b.q, 5.0).cuda()
    b.gpu(pkv, out=out)
    assert (out == 5.0).all()
    e = Trees([], [], 8, 2, seed=1)
    assert e.gpu(pkv).shape == (0, 8, D)
    expect_no_device_error(pkv)


# ---------------------------------------------------------------------------
# accepted paths
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("sizes,limit,vocab", [([1], 4, 5), ([26], 8, 3), ([0, 64, 1, 65, 0, 33], 16, 2), ([256, 255, 129], 40, 2), ([60] * 37, 1, 3),
                                              ([2] * 1000, 3, 2)])
def test_accept(pkv, sizes, limit, vocab):
    rng = np.random.default_rng(limit + len(sizes))
    words = -(-max(sizes) // 64) if max(sizes) else 1
    sees = [random_tree(n, rng, 4) for n in sizes]
    total = sum(sizes)
    target, draft = rng.integers(0, vocab, total), rng.integers(0, vocab, total)
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    mask = np.zeros((total, words), np.uint64)
    for s, n in enumerate(sizes):
        if n:
            mask[cu[s]:cu[s + 1]] = tr.words_of(sees[s], words)
    lens = np.array([n + int(rng.integers(0, 500)) for n in sizes], np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    path, count, follow, after = pkv.pkv_tree_accept(dev(target), dev(draft), dev(mask.view(np.int64)), dev(cu), dev(lens), max(sizes), limit)
    expect_no_device_error(pkv)
    assert follow.dtype == torch.int64 and path.dtype == count.dtype == after.dtype == torch.int32
    for s, n in enumerate(sizes):
        want, tok = tr.accept(target[cu[s]:cu[s + 1]], draft[cu[s]:cu[s + 1]], sees[s], limit)
        assert path[s].tolist() == want + [-1] * (limit - len(want))
        assert (count[s].item(), follow[s].item(), after[s].item()) == (len(want), tok, lens[s] - n + len(want))


def test_accept_leaves_out_bad_trees(pkv):
    dev = lambda a, t=torch.int32: torch.tensor(a, dtype=t).cuda()  # noqa: E731
    ids = torch.zeros(6, dtype=torch.int64).cuda()
    mask = torch.ones(6, 1, dtype=torch.int64).cuda()
    path, count, follow, after = pkv.pkv_tree_accept(ids, ids, mask, dev([0, 3, 6]), dev([2, 9]), 4, 2)
    assert pkv.pkv_get_device_error(clear=True) == (3, 0)
    assert path.tolist() == [[-1, -1], [0, 1]] and count.tolist() == [0, 2] and follow.tolist() == [-1, 0] and after.tolist() == [2, 8]
    pkv.pkv_tree_accept(ids, ids, mask, dev([0, 3, 7]), dev([5, 9]), 4, 2)
    assert pkv.pkv_get_device_error(clear=True) == (3, 1)


# ---------------------------------------------------------------------------
# rows moved and copied
# ---------------------------------------------------------------------------

class Pools:
    def __init__(self, layers, nb, block, hkv, fp8, seed):
        g = torch.Generator().manual_seed(seed)
        make = lambda shape, t: torch.randint(0, 256 if t is torch.uint8 else 2 ** 15, shape, generator=g).to(t)  # noqa: E731
        t = torch.uint8 if fp8 else torch.int16
        self.host = [[make((nb, block, hkv, D), t) for _ in range(layers)] for _ in "kv"]
        self.scales = [[make((nb, hkv, block), torch.uint8) for _ in range(layers)] for _ in "kv"] if fp8 else []
        kinds = (torch.float8_e4m3fn if fp8 else torch.bfloat16, torch.float8_e8m0fnu)
        self.dev = [[x.cuda() for x in y] for y in self.host + self.scales]
        self.views = [[x.view(kinds[i // 2]) for x in y] for i, y in enumerate(self.dev)]

    def move(self, moves):
        """(source block, row, destination block, row), in order, all read first."""
        for pool in self.host:
            for x in pool:
                kept = [x[b, r].clone() for b, r, _, _ in moves]
                for row, (_, _, b, r) in zip(kept, moves):
                    x[b, r] = row
        for pool in self.scales:
            for x in pool:
                kept = [x[b, :, r].clone() for b, r, _, _ in moves]
                for row, (_, _, b, r) in zip(kept, moves):
                    x[b, :, r] = row

    def check(self):
        for host, dev in zip(self.host + self.scales, self.dev):
            for x, y in zip(host, dev):
                assert torch.equal(x, y.cpu())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("layers,hkv,block", [(1, 1, 256), (3, 8, 256), (2, 3, 512), (128, 1, 256)])
def test_compact(pkv, layers, hkv, block, fp8):
    rng = np.random.default_rng(layers + hkv)
    nodes = [26, 1, 64, 0, 256, 9, 30]
    lens = [block + 10, 5, 64, 0, 2 * block - 3, block, block + 30]     # a path across a block's border, from its start, and to its end
    tables = np.full((7, 3), -1, np.int32)
    tables[:, :2] = rng.permutation(16)[:14].reshape(7, 2)
    paths = [sorted(rng.choice(n, size=min(n, c), replace=False)) if n else [] for n, c in zip(nodes, (9, 1, 20, 0, 200, 9, 5))]
    paths[6] = [0, 1, 2, 3, 29]
    width = 210
    path = np.full((7, width), -1, np.int32)
    for s, x in enumerate(paths):
        path[s, :len(x)] = x
    p = Pools(layers, 16, block, hkv, fp8, 3)
    pools = pkv.KvPools(*p.views)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    args = (dev(tables), dev(lens), dev(np.concatenate([[0], np.cumsum(nodes)])), dev(path), dev([len(x) for x in paths]))
    pkv.pkv_tree_compact(pools, *args)
    expect_no_device_error(pkv)
    moves = []
    for s, x in enumerate(paths):
        first = lens[s] - nodes[s]
        for d, i in enumerate(x):
            src, dst = first + i, first + d
            moves.append((tables[s, src // block], src % block, tables[s, dst // block], dst % block))
    p.move(moves)
    p.check()


def test_compact_refuses_bad_paths(pkv):
    dev = lambda a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    for path, count in (([0, 3, 2], 3), ([0, 5, 9], 3), ([-1, 1, 2], 3), ([0, 1, 2], 4), ([0, 2, 2], 3), ([0, 1, 2], -1)):
        p = Pools(2, 4, 256, 2, True, 1)
        pkv.pkv_tree_compact(pkv.KvPools(*p.views), dev([[0], [2]]), dev([40, 30]), dev([0, 9, 15]), dev([path, [0, 2, 5]]), dev([count, 3]))
        assert pkv.pkv_get_device_error(clear=True) == (9, 0), (path, count)
        p.move([(2, 24 + i, 2, 24 + d) for d, i in enumerate([0, 2, 5])])
        p.check()
    p = Pools(1, 4, 256, 2, False, 1)
    pkv.pkv_tree_compact(pkv.KvPools(*p.views), dev([[7]]), dev([40]), dev([0, 9]), dev([[0, 2, 5]]), dev([3]))
    assert pkv.pkv_get_device_error(clear=True) == (1, 0)
    pkv.pkv_tree_compact(pkv.KvPools(*p.views), dev([[1]]), dev([400]), dev([0, 9]), dev([[0, 2, 5]]), dev([3]))
    assert pkv.pkv_get_device_error(clear=True) == (3, 0)
    p.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
@pytest.mark.parametrize("layers,hkv,block", [(1, 1, 256), (3, 8, 256), (2, 3, 512), (128, 1, 256)])
def test_copy_blocks(pkv, layers, hkv, block, fp8):
    p = Pools(layers, 16, block, hkv, fp8, 4)
    pools = pkv.KvPools(*p.views)
    src, dst = [0, 1, -1, 0, 5, 6, 9], [10, 11, 12, 13, 14, 6, 15]
    rows = [block, 0, 7, 1, block - 1, 9, 37]
    dev = lambda a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    pkv.pkv_copy_blocks(pools, dev(src), dev(dst), dev(rows))
    expect_no_device_error(pkv)
    p.move([(s, r, d, r) for s, d, n in zip(src, dst, rows) if s >= 0 for r in range(n)])
    p.check()
    pkv.pkv_copy_blocks(pools, dev([3, 2]), dev([10, 12]))
    p.move([(s, r, d, r) for s, d in ((3, 10), (2, 12)) for r in range(block)])
    p.check()


def test_copy_blocks_records_bad_pairs(pkv):
    dev = lambda a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    p = Pools(2, 4, 256, 2, True, 1)
    pools = pkv.KvPools(*p.views)
    for src, dst, rows, code in ((4, 1, 3, 1), (0, -1, 3, 1), (0, 4, 3, 1), (0, 1, 257, 3), (0, 1, -1, 3)):
        pkv.pkv_copy_blocks(pools, dev([-5, src]), dev([2, dst]), dev([1, rows]))
        assert pkv.pkv_get_device_error(clear=True) == (code, 1)
        p.check()
    pkv.pkv_copy_blocks(pools, dev([]), dev([]))
    expect_no_device_error(pkv)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "8 bits"])
def test_a_step(pkv, fp8):
    """Draft, append, attend, sample, accept, compact, then decode: the cache is that of one-by-one decoding along the
    accepted path, and a sequence forked from it decodes alike."""
    rng = np.random.default_rng(21)
    g = torch.Generator().manual_seed(22)
    hq, hkv, block, nb, layers, vocab, base = 16, 8, 256, 12, 2, 50, 1.0e6
    nodes, before = [20, 7, 33], [250, 3, 500]
    lens = [b + n for b, n in zip(before, nodes)]
    sees = [random_tree(n, rng) for n in nodes]
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    total = int(cu[-1])
    tables = np.full((3, 3), -1, np.int32)
    perm = rng.permutation(nb)
    tables[0, :2], tables[1, :1], tables[2, :3] = perm[:2], perm[2:3], perm[3:6]
    dev = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a)).cuda() if t is None else torch.tensor(a, dtype=t).cuda()  # noqa: E731
    i32 = torch.int32
    if fp8:
        pool = lambda: [torch.zeros(nb, block, hkv, D, dtype=torch.uint8).cuda().view(torch.float8_e4m3fn) for _ in range(layers)]  # noqa: E731
        scale = lambda: [torch.full((nb, hkv, block), 127, dtype=torch.uint8).cuda().view(torch.float8_e8m0fnu) for _ in range(layers)]  # noqa: E731
        stores = (pool(), pool(), scale(), scale())
        append, attend, decode = pkv.pkv_rope_store_kvcache_fp8, pkv.pkv_tree_decode_fp8, pkv.pkv_decode_fp8
    else:
        pool = lambda: [torch.zeros(nb, block, hkv, D, dtype=torch.bfloat16).cuda() for _ in range(layers)]  # noqa: E731
        stores = (pool(), pool())
        append, attend, decode = pkv.pkv_rope_store_kvcache, pkv.pkv_tree_decode, pkv.pkv_decode
    randn = lambda *shape: torch.randn(*shape, generator=g).bfloat16().cuda()  # noqa: E731
    tab, cu_d, lens_d = dev(tables), dev(cu), dev(lens, i32)
    # the context
    ctx = sum(before)
    pos = torch.cat([torch.arange(b) for b in before]).to(i32).cuda()
    cu_ctx = dev(np.concatenate([[0], np.cumsum(before)]).astype(np.int32))
    slots = torch.empty(ctx, dtype=i32, device="cuda")
    pkv.pkv_slot_mapping(tab, nb, block, slots, cu_seqlens_q=cu_ctx, cu_seqlens_k=cu_ctx)
    for layer in range(layers):
        append(None, randn(ctx, hkv, D), randn(ctx, hkv, D), pos, slots, *[s[layer] for s in stores], base)
    # the drafts: rotated by depth, stored in node order
    mask = np.concatenate([tr.words_of(s, 1) for s in sees])
    mask_d = dev(mask.view(np.int64))
    depth = np.concatenate([s.sum(1) - 1 for s in sees])
    start = np.repeat(before, nodes)
    tree_pos, tree_slots = dev((start + depth).astype(np.int32)), torch.empty(total, dtype=i32, device="cuda")
    pkv.pkv_slot_mapping(tab, nb, block, tree_slots, cu_seqlens_q=cu_d, context_lens=lens_d)
    new = [(randn(total, hq, D), randn(total, hkv, D), randn(total, hkv, D)) for _ in range(layers)]
    outs = []
    for layer, (q, k, v) in enumerate(new):
        at = [s[layer] for s in stores]
        q = append(q, k, v, tree_pos, tree_slots, *at, base)
        outs.append(attend(q, *at, tab, lens_d, cu_d, mask_d, 33, max(lens), D ** -0.5))
    # sampled tokens decide the path: drafts are what was sampled at the parent, for about half of the nodes
    ids = pkv.pkv_sample(torch.randn(total, vocab, generator=g).cuda(), torch.ones(total).cuda(), seed=5)
    target = ids.cpu().numpy()
    parent = np.concatenate([[max([j for j in range(i) if s[i, j]], default=0) + c for i in range(len(s))] for s, c in zip(sees, cu)])
    draft = np.where(rng.random(total) < 0.7, target[parent], rng.integers(0, vocab, total))
    path, count, follow, after = pkv.pkv_tree_accept(ids, dev(draft), mask_d, cu_d, lens_d, 33, 16)
    pools = pkv.KvPools(*stores)
    pkv.pkv_tree_compact(pools, tab, lens_d, cu_d, path, count)
    expect_no_device_error(pkv)
    assert count.tolist() == [len(tr.accept(target[a:b], draft[a:b], s, 16)[0]) for a, b, s in zip(cu, cu[1:], sees)] and max(count.tolist()) > 2
    # one by one along the path, on a cache of its own
    single = [[x.view(torch.uint8).clone().view(x.dtype) for x in s] for s in stores]
    for s in range(3):
        for d in range(count[s].item()):
            i = int(cu[s]) + path[s, d].item()
            slot = dev([tables[s, (before[s] + d) // block] * block + (before[s] + d) % block], i32)
            one = dev([before[s] + d + 1], i32)
            for layer, (q, k, v) in enumerate(new):
                at = [x[layer] for x in single]
                q1 = append(q[i:i + 1], k[i:i + 1], v[i:i + 1], dev([before[s] + d], i32), slot, *at, base)
                o = decode(q1, *at, tab[s:s + 1], one, int(one), D ** -0.5)
                # two kernels' roundings of the same row: each within 2^-8 (|ref| + 2 A), A <= max|v| < 8
                assert (o[0].float() - outs[layer][i].float()).abs().max() < 0.1
    for a, b in zip(stores, single):
        for x, y in zip(a, b):
            for s in range(3):
                for p in range(after[s].item()):
                    blk, off = tables[s, p // block], p % block
                    pick = (lambda t: t.view(torch.uint8)[blk, off]) if x.dim() == 4 else (lambda t: t.view(torch.uint8)[blk, :, off])
                    assert torch.equal(pick(x), pick(y)), (s, p)
    # a fork of sequence 0: its full block shared, the last one copied
    last = (after[0].item() - 1) // block
    pkv.pkv_copy_blocks(pools, dev([tables[0, last]], i32), dev([perm[7]], i32), dev([after[0].item() - last * block], i32))
    fork = tables[0].copy()
    fork[last] = perm[7]
    q1 = randn(2, hq, D)
    q1[1] = q1[0]
    o = decode(q1, *[s[0] for s in stores], dev(np.stack([tables[0], fork])), dev([after[0].item()] * 2, i32), after[0].item(), D ** -0.5)
    assert (o[0].float() - o[1].float()).abs().max() < 0.05
    expect_no_device_error(pkv)
