"""The 8-bit KV cache on the GPU: appends, decode and prefill against float64.

Tolerances.  One rounding to bf16 is off by at most 2^-8 relative, to f16 2^-11, to e4m3 2^-4
(plus half its subnormal step, 2^-10 in units of the row's scale).  With A = sum_j p_j |v_j| per
output element:

* appends: V's codes and scales are exact.  A rotated K element carries the rotation's error of at
  most 1e-6 times its pair's length (hardware sine and cosine within 4e-7, three fp32
  roundings) before its one rounding; its scale is the definition's for a maximum that far off.
* decode: the weights are rounded to f16 (2^-11 A), scores and sums are fp32 (a score error of
  2^-13 would be 1000 roundings of a score near 1; 2^-13 A), the output to bf16 (2^-8 |ref|).
* prefill: bit for bit the bf16 prefill over the decoded cache; weights to bf16 (2^-8 A)."""
import numpy as np
import pytest
import torch

from oracle import fp8_cache as fc
from oracle import paged_attention as pa
from oracle import rope as rp
from pkv_testutil import expect_no_device_error

pytestmark = pytest.mark.gpu
D = 128


def e4m3(t):
    return t.view(torch.float8_e4m3fn)


def e8m0(t):
    return t.view(torch.float8_e8m0fnu)


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


class Cache:
    """A paged 8-bit cache with random rows where the sequences own positions and NaN codes and NaN
    scales everywhere else (free blocks, slots past a sequence's end)."""

    def __init__(self, kv_lens, hkv, block=256, seed=0, spread=3, width=None):
        rng = np.random.default_rng(seed)
        need = [-(-int(n) // block) for n in kv_lens]
        self.nb, self.block, self.hkv = sum(need) + 2, block, hkv
        perm = rng.permutation(self.nb)
        self.tables = np.full((len(need), width or max(max(need, default=1), 1)), -1, np.int32)
        self.k = np.full((self.nb, block, hkv, D), 0x7f, np.uint8)
        self.v = self.k.copy()
        self.ks = np.full((self.nb, hkv, block), 255, np.uint8)
        self.vs = self.ks.copy()
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = perm[at:at + n]
            for j in range(n):
                b, m = perm[at + j], min(block, int(kv_lens[s]) - j * block)
                for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
                    codes[b, :m] = fc.round_e4m3(np.clip(rng.normal(size=(m, hkv, D)) * 60, -448, 448))
                    scales[b, :, :m] = 121 + rng.integers(-spread, spread + 1, (hkv, m))
            at += n
        self.kv_lens = np.asarray(kv_lens, np.int32)

    def gpu(self):
        t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        return e4m3(t(self.k)), e4m3(t(self.v)), e8m0(t(self.ks)), e8m0(t(self.vs))

    def read(self, s):
        """Keys and values of sequence s, float64 [n, hkv, D]."""
        n = int(self.kv_lens[s])
        b = self.tables[s, :-(-n // self.block)]
        return tuple(fc.read_pool(c[b], sc[b]).reshape(-1, self.hkv, D)[:n] for c, sc in ((self.k, self.ks), (self.v, self.vs)))


def attention64(q, k, v, scale, mask=None):
    """q [m, hq, D], k and v [n, hkv, D] -> (out, A) [m, hq, D]; mask [m, n] of what each query sees."""
    G = q.shape[1] // k.shape[1]
    k, v = np.repeat(k, G, 1), np.repeat(v, G, 1)
    s = np.einsum("mhd,nhd->mhn", q, k) * scale
    if mask is not None:
        s = np.where(mask[:, None, :], s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    return np.einsum("mhn,nhd->mhd", p, v), np.einsum("mhn,nhd->mhd", p, np.abs(v))


def randn_bf16(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).bfloat16()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def make_pool(nb, bs, hkv, seed):
    rng = np.random.default_rng(seed)
    return [rng.integers(0, 120, (nb, bs, hkv, D), dtype=np.uint8), rng.integers(0, 120, (nb, bs, hkv, D), dtype=np.uint8),
            rng.integers(100, 140, (nb, hkv, bs), dtype=np.uint8), rng.integers(100, 140, (nb, hkv, bs), dtype=np.uint8)]


def on_gpu(pool):
    return [f(torch.from_numpy(a).cuda()) for f, a in zip((e4m3, e4m3, e8m0, e8m0), pool)]


def slots_for(n, nb, bs, seed, skip=False):
    slots = np.random.default_rng(seed).permutation(nb * bs)[:n].astype(np.int32)
    if skip:
        slots[1::3] = -1
    return slots


@pytest.mark.parametrize("n,hkv,bs,skip", [(1, 8, 256, False), (7, 1, 256, True), (33, 4, 512, True), (300, 16, 256, False)])
def test_store_is_the_definition_bit_for_bit(pkv, n, hkv, bs, skip):
    k, v = randn_bf16((n, hkv, D), 1), randn_bf16((n, hkv, D), 2, 30.0)
    k[0, 0] *= 2.0 ** -100
    v[0, -1] = 0
    v[-1, 0, 5] = 3e38
    pool = make_pool(3, bs, hkv, 3)
    slots = slots_for(n, 3, bs, 4, skip)
    got = on_gpu(pool)
    pkv.pkv_store_kvcache_fp8(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), *got)
    for x, codes, scales, gc, gs in ((k, pool[0], pool[2], got[0], got[2]), (v, pool[1], pool[3], got[1], got[3])):
        rc, rs = fc.store(codes, scales, x.double().numpy(), slots)
        assert np.array_equal(raw(gs), rs)
        assert np.array_equal(raw(gc), rc)
    expect_no_device_error(pkv)


def test_store_rows_with_infinities_and_nans_read_as_nan(pkv):
    k = randn_bf16((4, 2, D), 5)
    k[0, 0, 3], k[1, 1, 127], k[2, 0, 64] = float("inf"), float("nan"), -float("inf")
    pool = make_pool(1, 256, 2, 6)
    got = on_gpu(pool)
    slots = np.array([5, 6, 7, 8], np.int32)
    pkv.pkv_store_kvcache_fp8(k.cuda(), k.cuda(), torch.from_numpy(slots).cuda(), *got)
    for i, (codes, scales) in enumerate(((got[0], got[2]), (got[1], got[3]))):
        rc, rs = fc.store(pool[i], pool[2 + i], k.double().numpy(), slots)
        assert np.array_equal(raw(codes), rc) and np.array_equal(raw(scales), rs)
        assert (rs[0, 0, 5], rs[0, 1, 6], rs[0, 0, 7]) == (255, 255, 255)


def test_store_reads_views_of_a_fused_projection(pkv):
    n, hq, hkv = 21, 16, 4
    qkv = randn_bf16((n, (hq + 2 * hkv) * D + 8), 7).cuda()[:, : (hq + 2 * hkv) * D].unflatten(1, (hq + 2 * hkv, D))
    pool = make_pool(1, 256, hkv, 8)
    slots = torch.from_numpy(slots_for(n, 1, 256, 9)).cuda()
    a, b = on_gpu(pool), on_gpu(pool)
    pkv.pkv_store_kvcache_fp8(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], slots, *a)
    pkv.pkv_store_kvcache_fp8(qkv[:, hq:hq + hkv].contiguous(), qkv[:, hq + hkv:].contiguous(), slots, *b)
    for x, y in zip(a, b):
        assert np.array_equal(raw(x), raw(y))
    q_out = pkv.pkv_rope_store_kvcache_fp8(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:],
                                           torch.arange(n, dtype=torch.int32).cuda(), slots, *a, 1e6)
    ref = pkv.pkv_rope_store_kvcache_fp8(qkv[:, :hq].contiguous(), qkv[:, hq:hq + hkv].contiguous(), qkv[:, hq + hkv:].contiguous(),
                                         torch.arange(n, dtype=torch.int32).cuda(), slots, *b, 1e6)
    assert torch.equal(q_out, ref)
    for x, y in zip(a, b):
        assert np.array_equal(raw(x), raw(y))


@pytest.mark.parametrize("n,hq,hkv,far", [(1, 16, 8, False), (5, 8, 8, True), (40, 32, 4, True), (129, 8, 1, False)])
def test_rope_store_within_its_roundings(pkv, n, hq, hkv, far):
    q, k, v = randn_bf16((n, hq, D), 11), randn_bf16((n, hkv, D), 12, 4.0), randn_bf16((n, hkv, D), 13)
    pos = np.random.default_rng(14).integers(-2 ** 31 if far else 0, 2 ** 31 - 1 if far else 40000, n).astype(np.int32)
    pool = make_pool(2, 256, hkv, 15)
    slots = slots_for(n, 2, 256, 16, skip=n > 1)
    got = on_gpu(pool)
    base = 1e6
    q_rot = pkv.pkv_rope_store_kvcache_fp8(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(),
                                           torch.from_numpy(slots).cuda(), *got, base)
    pair = lambda x: np.tile(np.hypot(x[..., :64], x[..., 64:]), 2)  # noqa: E731
    ref_q = rp.rope(q.double().numpy(), pos, base)
    assert np.all(np.abs(q_rot.double().cpu().numpy() - ref_q) <= 2.0 ** -8 * np.abs(ref_q) + 1e-6 * pair(ref_q))
    # V and everything not written: exact
    rc, rs = fc.store(pool[1], pool[3], v.double().numpy(), slots)
    assert np.array_equal(raw(got[1]), rc) and np.array_equal(raw(got[3]), rs)
    ref_k = rp.rope(k.double().numpy(), pos, base)
    gc, gs = raw(got[0]), raw(got[2])
    written = np.zeros((2, 256), bool)
    for i, s in enumerate(slots):
        if s < 0:
            continue
        written[s // 256, s % 256] = True
        e = gs[s // 256, :, s % 256].astype(int) - 127
        x, err = ref_k[i], 1e-6 * pair(ref_k[i])
        amax, slack = np.abs(x).max(-1), err.max(-1)
        assert np.all(amax - slack <= 448 * 2.0 ** e) and np.all(amax + slack > 448 * 2.0 ** (e - 1.0))
        off = np.abs(fc.read_rows(gc[s // 256, s % 256], gs[s // 256, :, s % 256]) - x)
        assert np.all(off <= (2.0 ** -4 * np.abs(x) + 2.0 ** (e - 10.0)[:, None]) + err * 1.1)
    assert np.array_equal(gc[~written], pool[0][~written])
    assert np.array_equal(gs.swapaxes(1, 2)[~written], pool[2].swapaxes(1, 2)[~written])
    expect_no_device_error(pkv)


def test_rope_store_in_place_and_without_q(pkv):
    n = 19
    q, k, v = (randn_bf16((n, h, D), s).cuda() for h, s in ((16, 21), (8, 22), (8, 23)))
    pos, slots = torch.arange(n, dtype=torch.int32).cuda(), torch.from_numpy(slots_for(n, 1, 256, 24)).cuda()
    pool = make_pool(1, 256, 8, 25)
    a, b = on_gpu(pool), on_gpu(pool)
    ref = pkv.pkv_rope_store_kvcache_fp8(q, k, v, pos, slots, *a, 1e4)
    assert pkv.pkv_rope_store_kvcache_fp8(None, k, v, pos, slots, *b, 1e4) is None
    for x, y in zip(a, b):
        assert np.array_equal(raw(x), raw(y))
    here = q.clone()
    assert pkv.pkv_rope_store_kvcache_fp8(here, k, v, pos, slots, *b, 1e4, q_out=here) is here
    assert torch.equal(here, ref)
    # the same rotation as the bf16 append's, to a rounding
    kc = torch.zeros(1, 256, 8, D, dtype=torch.bfloat16, device="cuda")
    other = pkv.pkv_rope_store_kvcache(q, k, v, pos, slots, kc, torch.zeros_like(kc), 1e4).double()
    assert torch.all((ref.double() - other).abs() <= 2.0 ** -7 * other.abs() + 2e-6 * q.double().abs().amax())


@pytest.mark.parametrize("n,hq,hkv", [(2500, 16, 8), (5001, 8, 1), (1700, 32, 8), (5003, 3, 2), (4900, 0, 8)])
def test_many_tokens_at_once_are_the_same_as_a_few_at_a_time(pkv, n, hq, hkv):
    """Large appends take a kernel of their own (more work than four items for every warp of the GPU): bit for
    bit what appends of 400 tokens write, from views of a fused projection, with skipped rows."""
    g = torch.Generator().manual_seed(n)
    width = (hq + 2 * hkv) * D
    qkv = (torch.randn(n, width + 24, generator=g) * 3).bfloat16().cuda()[:, :width].unflatten(1, (hq + 2 * hkv, D))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = torch.randint(0, 2 ** 20, (n,), generator=g, dtype=torch.int32).cuda()
    nb = -(-n // 256) + 1
    slots = torch.from_numpy(slots_for(n, nb, 256, n + 1, skip=True)).cuda()
    pool = make_pool(nb, 256, hkv, n + 2)
    a, b = on_gpu(pool), on_gpu(pool)
    parts = [slice(i, i + 400) for i in range(0, n, 400)]
    if hq:
        once = pkv.pkv_rope_store_kvcache_fp8(q, k, v, pos, slots, *a, 1e6)
        few = torch.cat([pkv.pkv_rope_store_kvcache_fp8(q[x], k[x], v[x], pos[x], slots[x], *b, 1e6) for x in parts])
        assert torch.equal(once, few)
    else:
        pkv.pkv_store_kvcache_fp8(k, v, slots, *a)
        for x in parts:
            pkv.pkv_store_kvcache_fp8(k[x], v[x], slots[x], *b)
    for x, y, old in zip(a, b, pool):
        assert np.array_equal(raw(x), raw(y)) and not np.array_equal(raw(x), old)
    if hq:                                                # and without q, and in place
        c = on_gpu(pool)
        assert pkv.pkv_rope_store_kvcache_fp8(None, k, v, pos, slots, *c, 1e6) is None
        for x, y in zip(a, c):
            assert np.array_equal(raw(x), raw(y))
        pkv.pkv_rope_store_kvcache_fp8(q, k, v, pos, slots, *c, 1e6, q_out=q)
        assert torch.equal(once, q)
    expect_no_device_error(pkv)


def test_store_slot_past_the_pool_is_skipped_and_recorded(pkv):
    k = randn_bf16((3, 8, D), 31).cuda()
    pool = make_pool(1, 256, 8, 32)
    got = on_gpu(pool)
    pkv.pkv_store_kvcache_fp8(k, k, torch.tensor([256, -1, 2 ** 31 - 1], dtype=torch.int32).cuda(), *got)
    code, info = pkv.pkv_get_device_error(clear=True)
    assert code == 2 and info in (0, 2)
    for a, b in zip(pool, got):
        assert np.array_equal(a, raw(b))


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

def decode_case(pkv, kv_lens, hq, hkv, block=256, seed=0, spread=3, q_std=1.5, scale=D ** -0.5, check=None):
    c = Cache(kv_lens, hkv, block, seed, spread)
    q = randn_bf16((len(kv_lens), hq, D), seed + 1, q_std)
    out = torch.full((len(kv_lens), hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    args = (q.cuda(), *c.gpu(), torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.kv_lens).cuda(), int(max(kv_lens)), scale)
    pkv.pkv_decode_fp8(*args, out=out)
    got = out.double().cpu().numpy()
    for b in (range(len(kv_lens)) if check is None else check):
        if kv_lens[b] == 0:
            assert not got[b].any()
            continue
        ref, A = attention64(q[b:b + 1].double().numpy(), *c.read(b), scale)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * A + 1e-30
        assert np.all(np.abs(got[b:b + 1] - ref) <= tol), (b, kv_lens[b], float((np.abs(got[b:b + 1] - ref) / tol).max()))
    expect_no_device_error(pkv)
    return args, out


@pytest.mark.parametrize("hq,hkv", [(16, 16), (16, 8), (16, 4), (32, 4), (8, 1)])
def test_decode_groups_and_lengths(pkv, hq, hkv):
    """Lengths around the 32-token chunk and the block, empty sequences first, between and last."""
    decode_case(pkv, [0, 1, 2, 31, 32, 33, 0, 63, 64, 65, 255, 256, 257, 300, 511, 512, 513, 0], hq, hkv, seed=hq * 10 + hkv)


@pytest.mark.parametrize("kv_lens,hq,hkv,block", [([1], 16, 8, 256), ([5000], 8, 1, 512), ([3000, 1, 0, 1700], 32, 4, 1024),
                                                  ([700] * 40, 16, 8, 256)])
def test_decode_few_and_many_pieces(pkv, kv_lens, hq, hkv, block):
    decode_case(pkv, kv_lens, hq, hkv, block, seed=len(kv_lens), check=[0, len(kv_lens) - 1])


def test_decode_rows_of_very_different_scale(pkv):
    """Rows' scales spread over 2^80: the weights' reference follows the largest weight times scale."""
    decode_case(pkv, [40, 300, 513], 16, 8, seed=51, spread=40, q_std=2.0 ** -10)
    decode_case(pkv, [40, 300], 16, 8, seed=52, spread=40, q_std=2.0 ** -45)


def test_decode_peaked_and_growing_scores(pkv):
    """Large queries: softmax concentrated on few keys, the running maximum moving along the context."""
    decode_case(pkv, [2000, 333], 16, 4, seed=53, q_std=40.0)


def test_decode_zero_rows(pkv):
    """All-zero V rows (scale exponent -126) and all-zero K rows beside ordinary ones."""
    c = Cache([100, 40], 8, seed=54)
    for s, n in ((0, 100), (1, 40)):
        b = c.tables[s, 0]
        zero = np.arange(n) % 3 == 0 if s == 0 else np.ones(n, bool)
        c.v[b, :n][zero], c.vs[b, :, np.nonzero(zero)[0]] = 0, 1
        c.k[b, :n][::5], c.ks[b, :, :n][:, ::5] = 0, 1
    q = randn_bf16((2, 16, D), 55)
    out = pkv.pkv_decode_fp8(q.cuda(), *c.gpu(), torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.kv_lens).cuda(), 100, D ** -0.5)
    ref, A = attention64(q[:1].double().numpy(), *c.read(0), D ** -0.5)
    assert np.all(np.abs(out[:1].double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * A)
    assert not out[1].any()


def test_decode_nan_rows_show(pkv):
    """A K row or a V row that reads as NaN makes its sequence's heads NaN and nobody else's."""
    c = Cache([70, 70, 70], 8, seed=56)
    c.ks[c.tables[0, 0], 2, 40] = 255
    c.vs[c.tables[2, 0], 5, 3] = 255
    q = randn_bf16((3, 16, D), 57)
    out = pkv.pkv_decode_fp8(q.cuda(), *c.gpu(), torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.kv_lens).cuda(), 70, D ** -0.5)
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros_like(nan)
    want[0, 4:6] = want[2, 10:12] = True
    assert np.array_equal(nan, want)


def test_decode_repeats_bit_for_bit_on_any_stream_and_in_a_graph(pkv):
    args, out = decode_case(pkv, [900, 17, 0, 2500, 333], 16, 8, seed=58)
    ws = pkv.decode_fp8_workspace(5, 16, 8, D)
    ws.fill_(0xff)                                        # nothing in the workspace needs to start at zero
    other = torch.empty_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.pkv_decode_fp8(*args, out=other, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_decode_fp8(*args, out=other, workspace=ws)
    other.fill_(0)
    graph.replay()
    assert torch.equal(out, other)
    lens = args[6]                                        # other lengths in the same buffers
    lens.copy_(torch.tensor([1, 17, 400, 2000, 0], dtype=torch.int32))
    ref = pkv.pkv_decode_fp8(*args)
    graph.replay()
    assert torch.equal(ref[[0, 1, 3, 4]], other[[0, 1, 3, 4]])
    pkv.pkv_get_device_error(clear=True)                  # sequence 2 had no blocks: recorded


def test_decode_bad_block_and_length_are_recorded(pkv):
    c = Cache([300, 40], 8, seed=59)
    c.tables[0, 1] = c.nb
    q = randn_bf16((2, 16, D), 60).cuda()
    run = lambda lens: pkv.pkv_decode_fp8(q, *c.gpu(), torch.from_numpy(c.tables).cuda(),  # noqa: E731
                                          torch.tensor(lens, dtype=torch.int32).cuda(), 300, D ** -0.5)
    out = run([300, 40])
    assert pkv.pkv_get_device_error(clear=True) == (1, 0)
    ref, A = attention64(q[1:].double().cpu().numpy(), *c.read(1), D ** -0.5)
    assert np.all(np.abs(out[1:].double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * A)
    out = run([-5, 40])
    assert pkv.pkv_get_device_error(clear=True) == (3, 0) and not out[0].any()


def test_decode_refusals(pkv):
    c = Cache([40], 8, seed=61)
    q = randn_bf16((1, 16, D), 62).cuda()
    k, v, ks, vs = c.gpu()
    bt, ln = torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.kv_lens).cuda()
    with pytest.raises(TypeError):
        pkv.pkv_decode_fp8(q, k.view(torch.uint8), v, ks, vs, bt, ln, 40, 0.1)
    with pytest.raises(ValueError):
        pkv.pkv_decode_fp8(q, k, v, ks.transpose(1, 2).contiguous(), vs, bt, ln, 40, 0.1)
    with pytest.raises(ValueError):
        pkv.pkv_decode_fp8(q, k, v, ks, vs, bt, torch.cat([ln, ln]), 40, 0.1)
    with pytest.raises(ValueError):
        pkv.pkv_decode_fp8(q, k, v, ks, vs, bt, ln, 40, 0.1, out=torch.empty(2, 16, D, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(pkv.PkvError):
        pkv.pkv_decode_fp8(q, k, v, ks, vs, bt, ln, 40, 0.1, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pkv.PkvError):
        pkv.pkv_decode_fp8(q, k, v, ks, vs, bt, ln, 40, -0.1)


# ---------------------------------------------------------------------------
# prefill
# ---------------------------------------------------------------------------

def prefill_case(pkv, q_lens, kv_lens, hq, hkv, block=256, seed=0, check=None, q_std=1.5):
    c = Cache(kv_lens, hkv, block, seed)
    ql = np.asarray(q_lens, np.int32)
    cu = lambda a: torch.from_numpy(np.concatenate([[0], np.cumsum(a)]).astype(np.int32)).cuda()  # noqa: E731
    q = randn_bf16((int(ql.sum()), hq, D), seed + 1, q_std)
    scale = D ** -0.5
    pools = c.gpu()
    bt = torch.from_numpy(c.tables).cuda()
    args = (q.cuda(), *pools, cu(ql), cu(c.kv_lens), bt, int(ql.max()), int(c.kv_lens.max()), int(c.kv_lens.sum()), scale)
    out = pkv.pkv_prefill_varlen_fp8(*args)
    # the decoded cache, exact in bf16, through the bf16 prefill
    decoded = [torch.from_numpy(fc.read_pool(a, s)).bfloat16().cuda() for a, s in ((c.k, c.ks), (c.v, c.vs))]
    same = pkv.pkv_prefill_varlen(q.cuda(), *decoded, cu(ql), cu(c.kv_lens), bt, int(ql.max()), int(c.kv_lens.max()), scale)
    assert torch.equal(out.view(torch.int16), same.view(torch.int16))
    got = out.double().cpu().numpy()
    at = np.concatenate([[0], np.cumsum(ql)])
    for s in (range(len(ql)) if check is None else check):
        n, m = int(c.kv_lens[s]), int(ql[s])
        if m == 0:
            continue
        rows = slice(at[s], at[s + 1])
        ref, A = attention64(q[rows].double().numpy(), *c.read(s), scale, np.tril(np.ones((m, n), bool), n - m))
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -13) * A
        assert np.all(np.abs(got[rows] - ref) <= tol), (s, m, n)
    expect_no_device_error(pkv)
    return args, out


@pytest.mark.parametrize("hq,hkv", [(16, 16), (16, 8), (16, 4), (32, 4), (8, 1)])
def test_prefill_groups_and_lengths(pkv, hq, hkv):
    prefill_case(pkv, [1, 5, 0, 33, 128, 1, 100], [1, 5, 40, 129, 128, 256, 300], hq, hkv, seed=hq * 7 + hkv)


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,block", [([1], [1], 16, 8, 256), ([37], [293], 16, 8, 256),
                                                        ([700, 3], [700, 1025], 8, 1, 512), ([257] * 9, [257] * 9, 16, 8, 1024)])
def test_prefill_few_and_many(pkv, q_lens, kv_lens, hq, hkv, block):
    prefill_case(pkv, q_lens, kv_lens, hq, hkv, block, seed=len(q_lens), check=[0, len(q_lens) - 1])


def test_prefill_workspace_reused_and_captured(pkv):
    args, out = prefill_case(pkv, [60, 200], [300, 200], 16, 8, seed=71)
    ws = pkv.prefill_fp8_workspace(2, 16, 8, D, 200, 300, 500)
    ws.fill_(0xff)
    other = torch.empty_like(out)
    pkv.pkv_prefill_varlen_fp8(*args, out=other, workspace=ws)
    assert torch.equal(out, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_prefill_varlen_fp8(*args, out=other, workspace=ws)
    for _ in range(2):
        other.fill_(0)
        graph.replay()
        assert torch.equal(out, other)


def test_prefill_total_too_small_is_recorded(pkv):
    """A batch that does not fit total_k: the sequences that fit are right, the other is recorded."""
    args, out = prefill_case(pkv, [60, 200, 50], [300, 200, 250], 16, 8, seed=72)
    args = (*args[:10], 500, args[11])
    got = pkv.pkv_prefill_varlen_fp8(*args)
    assert pkv.pkv_get_device_error(clear=True) == (3, 2)
    assert torch.equal(got[:260], out[:260])


def test_prefill_bad_block_is_recorded(pkv):
    args, out = prefill_case(pkv, [60, 200], [300, 200], 16, 8, seed=73)
    bt = args[7].clone()
    bt[0, 1] = 10 ** 6
    got = pkv.pkv_prefill_varlen_fp8(*args[:7], bt, *args[8:])
    assert pkv.pkv_get_device_error(clear=True) == (1, 0)
    assert torch.equal(got[60:], out[60:])


# ---------------------------------------------------------------------------
# sharing, sizes and streams
# ---------------------------------------------------------------------------

def test_calls_of_different_batches_share_a_workspace_in_stream_order(pkv):
    """Two batches of other lengths, tables and sizes in turn on one workspace with nothing waited for between
    them: each call's plan, tiles and pieces are its own."""
    a = prefill_case(pkv, [60, 200, 1], [300, 200, 513], 16, 8, seed=91)
    b = prefill_case(pkv, [257, 3], [257, 1000], 16, 8, seed=92)
    n = max(pkv.pkv_prefill_fp8_workspace_size(len(x[0][5]) - 1, 16, 8, D, *x[0][8:11]) for x in (a, b))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    got = [pkv.pkv_prefill_varlen_fp8(*x[0], workspace=ws) for _ in range(10) for x in (a, b)]
    for i, o in enumerate(got):
        assert torch.equal(o, (a, b)[i % 2][1])
    c = decode_case(pkv, [900, 17, 0, 2500, 333], 16, 8, seed=93)
    d = decode_case(pkv, [31] * 40, 16, 8, seed=94, check=[0])
    ws = pkv.decode_fp8_workspace(40, 16, 8, D)
    got = [pkv.pkv_decode_fp8(*x[0], workspace=ws) for _ in range(10) for x in (c, d)]
    for i, o in enumerate(got):
        assert torch.equal(o, (c, d)[i % 2][1])


def test_calls_on_two_streams_at_once_with_their_own_workspaces(pkv):
    a = decode_case(pkv, [3000, 17, 0, 2500, 333], 16, 8, seed=95)
    b = prefill_case(pkv, [257, 300], [257, 1000], 16, 8, seed=96)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):                                   # workspaces and outputs allocated by the calls themselves
        outs.append((pkv.pkv_decode_fp8(*a[0], stream=s1), pkv.pkv_prefill_varlen_fp8(*b[0], stream=s2)))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, a[1]) and torch.equal(y, b[1])


def test_decode_largest_batch(pkv):
    """4096 sequences of 0 to 3 tokens sharing one block; one more is refused."""
    c = Cache([3], 2, seed=97)
    B = 4096
    lens = np.arange(B) % 4
    q = randn_bf16((B, 4, D), 98)
    args = (*c.gpu(), torch.full((B + 1, 1), int(c.tables[0, 0]), dtype=torch.int32).cuda())
    out = pkv.pkv_decode_fp8(q.cuda(), *args[:4], args[4][:B], torch.from_numpy(lens.astype(np.int32)).cuda(), 3, D ** -0.5)
    k, v = c.read(0)
    got = out.double().cpu().numpy()
    for n in (1, 2, 3):
        rows = np.nonzero(lens == n)[0]
        ref, A = attention64(q[rows].double().numpy(), k[:n], v[:n], D ** -0.5)
        assert np.all(np.abs(got[rows] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * A)
    assert not got[lens == 0].any()
    with pytest.raises(pkv.PkvError):
        pkv.pkv_decode_fp8(torch.cat([q, q[:1]]).cuda(), *args, torch.ones(B + 1, dtype=torch.int32).cuda(), 3, D ** -0.5)
    expect_no_device_error(pkv)


def test_empty_calls_do_nothing(pkv):
    pool = on_gpu(make_pool(1, 256, 8, 99))
    z = torch.zeros(0, 8, D, dtype=torch.bfloat16, device="cuda")
    zq = torch.zeros(0, 16, D, dtype=torch.bfloat16, device="cuda")
    zi = torch.zeros(0, dtype=torch.int32, device="cuda")
    pkv.pkv_store_kvcache_fp8(z, z, zi, *pool)
    assert pkv.pkv_rope_store_kvcache_fp8(zq, z, z, zi, zi, *pool, 1e4).shape == (0, 16, D)
    assert pkv.pkv_decode_fp8(zq, *pool, torch.zeros(0, 1, dtype=torch.int32, device="cuda"), zi, 0, 0.1).shape == (0, 16, D)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert pkv.pkv_prefill_varlen_fp8(zq, *pool, cu, cu, torch.zeros(2, 1, dtype=torch.int32, device="cuda"), 0, 0, 0, 0.1).shape == (0, 16, D)
    assert pkv.pkv_sample_filtered(torch.zeros(0, 50, device="cuda"), torch.zeros(0, device="cuda"), None, None, None, 1).shape == (0,)
    expect_no_device_error(pkv)


def test_prefill_of_more_sequences_than_fit_near(pkv):
    """1100 one-token prompts: more running counts than the decoding kernel keeps in shared memory."""
    prefill_case(pkv, [1] * 1100, [1 + i % 3 for i in range(1100)], 8, 1, seed=90, check=list(range(0, 1100, 97)))


# ---------------------------------------------------------------------------
# together: a prompt with a cached prefix, then decode steps, then sampling
# ---------------------------------------------------------------------------

def test_a_serving_run_on_the_8_bit_cache(pkv):
    """Prompts appended (rotated) and attended, then three decode steps that append, attend and sample,
    each against float64 over the cache the oracle keeps."""
    hq, hkv, block, base, scale = 16, 8, 256, 1e6, D ** -0.5
    kv = np.array([260, 31, 511], np.int32)
    B, width, nb = 3, 3, 12
    tables = np.random.default_rng(81).permutation(nb)[: B * width].reshape(B, width).astype(np.int32)
    bt = torch.from_numpy(tables).cuda()
    pool = [np.full((nb, block, hkv, D), 0x7f, np.uint8) for _ in range(2)] + [np.full((nb, hkv, block), 255, np.uint8) for _ in range(2)]
    cache = on_gpu(pool)

    def read(s, n):
        b = tables[s, :-(-n // block)]
        return tuple(fc.read_pool(raw(cache[i])[b], raw(cache[2 + i])[b]).reshape(-1, hkv, D)[:n] for i in range(2))

    def append(q, k, v, pos, slots):
        return pkv.pkv_rope_store_kvcache_fp8(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(pos.astype(np.int32)).cuda(), slots, *cache, base)

    done = np.zeros(B, np.int32)
    for chunk in (np.array([256, 20, 300], np.int32), kv - np.array([256, 20, 300], np.int32)):     # the second chunk has a cached prefix
        now = done + chunk
        cu_q, cu_k = (torch.from_numpy(np.concatenate([[0], np.cumsum(a)]).astype(np.int32)).cuda() for a in (chunk, now))
        n = int(chunk.sum())
        q, k, v = (randn_bf16((n, h, D), int(done.sum()) + 82 + i) for i, h in enumerate((hq, hkv, hkv)))
        slots = torch.empty(n, dtype=torch.int32, device="cuda")
        pkv.pkv_slot_mapping(bt, nb, block, slots, cu_seqlens_q=cu_q, cu_seqlens_k=cu_k)
        pos = np.concatenate([np.arange(a, b) for a, b in zip(done, now)])
        q_rot = append(q, k, v, pos, slots)
        out = pkv.pkv_prefill_varlen_fp8(q_rot, *cache, cu_q, cu_k, bt, int(chunk.max()), int(now.max()), int(now.sum()), scale)
        at = np.concatenate([[0], np.cumsum(chunk)])
        for s in range(B):
            kk, vv = read(s, int(now[s]))
            fresh = rp.rope(k[at[s]:at[s + 1]].double().numpy(), pos[at[s]:at[s + 1]], base)
            assert np.all(np.abs(kk[done[s]:] - fresh) <= 2.0 ** -4 * np.abs(fresh) + 2.0 ** -9 * np.abs(fresh).max(-1, keepdims=True))
            m = int(chunk[s])
            ref, A = attention64(q_rot[at[s]:at[s + 1]].double().cpu().numpy(), kk, vv, scale, np.tril(np.ones((m, int(now[s])), bool), int(now[s]) - m))
            assert np.all(np.abs(out[at[s]:at[s + 1]].double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -13) * A)
        done = now
    for step in range(3):
        ctx = done + 1
        lens = torch.from_numpy(ctx).cuda()
        q, k, v = (randn_bf16((B, h, D), 900 + 10 * step + i) for i, h in enumerate((hq, hkv, hkv)))
        slots = torch.empty(B, dtype=torch.int32, device="cuda")
        pkv.pkv_slot_mapping(bt, nb, block, slots, context_lens=lens)
        q_rot = append(q, k, v, done, slots)
        out = pkv.pkv_decode_fp8(q_rot, *cache, bt, lens, int(ctx.max()), scale)
        for s in range(B):
            ref, A = attention64(q_rot[s:s + 1].double().cpu().numpy(), *read(s, int(ctx[s])), scale)
            assert np.all(np.abs(out[s:s + 1].double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * A)
        head = randn_bf16((hq * D, 4001), 990).cuda().float() * 0.03
        logits = out.float().view(B, -1) @ head
        T, tk, tp, mp = (torch.tensor(a).cuda() for a in ([0.8, 1.0, 0.6], [40, 0, 7], [0.9, 0.8, 1.0], [0.0, 0.02, 0.0]))
        ids = pkv.pkv_sample_filtered(logits, T, tk.int(), tp, mp, seed=5, offset=B * step)
        from oracle import filtered as fl
        ref, clear = fl.decided(logits.double().cpu().numpy(), T.double().cpu().numpy(), tk.cpu().numpy(), tp.double().cpu().numpy(),
                                      mp.double().cpu().numpy(), 5, B * step)
        assert np.array_equal(ids.cpu().numpy()[clear], ref[clear]) and clear.sum() >= 2
        done = ctx
    expect_no_device_error(pkv)


def test_a_tensor_on_another_device_is_refused_wherever_it_is(pkv):
    c = Cache([40], 2, seed=91)
    k, v, ks, vs = c.gpu()
    bt, ln = torch.from_numpy(c.tables).cuda(), torch.from_numpy(c.kv_lens).cuda()
    q, kv = randn_bf16((1, 4, D), 92).cuda(), randn_bf16((1, 2, D), 93).cuda()
    one, cu_q, cu_k = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, 1]).int().cuda(), torch.tensor([0, 40]).int().cuda()
    logits, row = torch.zeros(1, 9, device="cuda"), torch.ones(1, device="cuda")
    calls = [(pkv.pkv_store_kvcache_fp8, [kv, kv, one, k, v, ks, vs], []),
             (pkv.pkv_rope_store_kvcache_fp8, [q, kv, kv, one, one, k, v, ks, vs], [1e4]),
             (pkv.pkv_decode_fp8, [q, k, v, ks, vs, bt, ln], [40, 0.1]),
             (pkv.pkv_prefill_varlen_fp8, [q, k, v, ks, vs, cu_q, cu_k, bt], [1, 40, 40, 0.1]),
             (pkv.pkv_sample_filtered, [logits, row, one, row, row], [1])]
    for f, tensors, rest in calls:
        f(*tensors, *rest)
        for i in range(len(tensors)):
            with pytest.raises(ValueError):
                f(*(t.cpu() if j == i else t for j, t in enumerate(tensors)), *rest)
    expect_no_device_error(pkv)
