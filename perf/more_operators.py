"""Decoding along a tree of drafted tokens over the paged KV cache: cases, inputs and plain forms.

A step drafts several tokens per sequence, arranged in a tree: node 0 is the token that is
certain, every other node a guess at what follows its parent.  All nodes' K/V rows are in the
cache, at the sequence's last positions, and the tree is given by one bit mask per node: bit j
of node i says that i sees node j (its ancestors and itself).

  tree      attention of the nodes over the sequence's context and their ancestors
  accept    the path from node 0 along which each draft is what the model sampled at its parent
  compact   the accepted path's rows, moved together in every layer's pools
  copy      the filled rows of blocks copied to other blocks in every layer's pools (a fork)

on a bf16 cache and on the 8-bit one (128 e4m3 codes and a power-of-two scale per row).
`own` chooses between the plain forms here (elementary torch operations) and the library's
kernels.
"""
import math

import numpy as np
import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")

D = 128
SHAPES = ((16, 8), (16, 16), (16, 4), (32, 4), (8, 1), (32, 8))     # query heads, KV heads
MOST_KEYS = 230000            # keys of a batch, with 8 KV heads
MOST_PAIRS = 230000 * 64 * 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one conversation, a handful of drafts: latency
        {"name": "tree one sequence", "kind": "tree", "batch": 1, "lo": 611, "hi": 611, "n_lo": 8, "n_hi": 8, "lens": 1, "hq": 16, "hkv": 8, "block": 256, "fp8": False},
        # a serving batch with small trees, 512 to 4096 tokens of context
        {"name": "tree batch of 64", "kind": "tree", "batch": 64, "lo": 512, "hi": 4096, "n_lo": 12, "n_hi": 16, "lens": 2, "hq": 16, "hkv": 8, "block": 256, "fp8": False},
        # large trees of uneven size on short contexts, four query heads to a KV head: the most work per byte
        {"name": "tree large trees", "kind": "tree", "batch": 32, "lo": 80, "hi": 2999, "n_lo": 33, "n_hi": 64, "lens": 3, "hq": 32, "hkv": 8, "block": 256, "fp8": False},
        # long documents: few sequences, so each is split over its length
        {"name": "tree long contexts", "kind": "tree", "batch": 8, "lo": 16384, "hi": 40960, "n_lo": 60, "n_hi": 60, "lens": 4, "hq": 16, "hkv": 8, "block": 256, "fp8": False},
        # the serving batch on the 8-bit cache
        {"name": "tree batch of 64, 8 bits", "kind": "tree", "batch": 64, "lo": 512, "hi": 4096, "n_lo": 12, "n_hi": 16, "lens": 2, "hq": 16, "hkv": 8, "block": 256, "fp8": True},
        # long documents on the 8-bit cache, eight query heads to a KV head, an odd tree
        {"name": "tree long contexts, 8 bits", "kind": "tree", "batch": 7, "lo": 16384, "hi": 40960, "n_lo": 13, "n_hi": 29, "lens": 5, "hq": 32, "hkv": 4, "block": 512, "fp8": True},
        # one conversation's drafts after the model has sampled at each: latency
        {"name": "accept one sequence", "kind": "accept", "batch": 1, "n_lo": 26, "n_hi": 26, "path": 8, "lens": 6},
        # a large batch of large trees, uneven, some of them empty
        {"name": "accept 512 sequences", "kind": "accept", "batch": 512, "n_lo": 0, "n_hi": 64, "path": 16, "lens": 7},
        # one conversation's accepted rows in all layers: latency
        {"name": "compact one sequence", "kind": "compact", "batch": 1, "layers": 28, "n_lo": 26, "n_hi": 26, "path": 8, "lens": 8, "hkv": 8, "block": 256, "fp8": False},
        # a serving batch on the 8-bit cache
        {"name": "compact 128 sequences, 8 bits", "kind": "compact", "batch": 128, "layers": 28, "n_lo": 1, "n_hi": 64, "path": 12, "lens": 9, "hkv": 8, "block": 256, "fp8": True},
        # one sequence forks: its last block, partly filled, in all layers
        {"name": "copy one block", "kind": "copy", "pairs": 1, "layers": 28, "r_lo": 137, "r_hi": 137, "lens": 10, "hkv": 8, "block": 256, "fp8": False},
        # many samples of many prompts start on the 8-bit cache, blocks filled to any row
        {"name": "copy 64 blocks, 8 bits", "kind": "copy", "pairs": 64, "layers": 28, "r_lo": 0, "r_hi": 256, "lens": 11, "hkv": 8, "block": 256, "fp8": True},
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, math.floor(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(("tree", "tree", "tree", "accept", "compact", "copy"))
    hq, hkv = rng.choice(SHAPES)
    block = rng.choice((256, 256, 512))
    fp8 = rng.random() < 0.5
    lens = rng.randrange(1 << 30)
    if kind == "tree":
        batch = _log_int(rng, 1, 256)
        n = _log_int(rng, 1, 256)
        hi = max(n, _log_int(rng, 1, max(1, min(40960, MOST_KEYS * 8 // hkv // batch, MOST_PAIRS // (n * hq * batch)))))
        if hi * batch * n * hq > MOST_PAIRS:
            batch = max(1, MOST_PAIRS // (hi * n * hq))
        return {"kind": kind, "batch": batch, "lo": rng.randint(0 if batch > 4 else 1, hi), "hi": hi, "n_lo": rng.randint(1, n), "n_hi": n,
                "lens": lens, "hq": hq, "hkv": hkv, "block": block, "fp8": fp8}
    n = _log_int(rng, 1, 256)
    if kind == "accept":
        return {"kind": kind, "batch": _log_int(rng, 1, 32768 // n if n > 64 else 512), "n_lo": rng.randint(0, n), "n_hi": n, "path": _log_int(rng, 1, 32), "lens": lens}
    layers = _log_int(rng, 1, 48)
    if kind == "compact":
        most = max(1, int(3.6e9 // (layers * 2 * 2 * block * hkv * D * 2)))
        return {"kind": kind, "batch": min(most, _log_int(rng, 1, 256)), "layers": layers, "n_lo": rng.randint(1, n), "n_hi": n, "path": _log_int(rng, 1, 32),
                "lens": lens, "hkv": hkv, "block": block, "fp8": fp8}
    most = max(1, int(3.6e9 // (layers * 2 * 2 * block * hkv * D * 2)))
    hi = rng.randint(1, block)
    return {"kind": kind, "pairs": min(most, _log_int(rng, 1, 64)), "layers": layers, "r_lo": rng.randint(0, hi), "r_hi": hi, "lens": lens,
            "hkv": hkv, "block": block, "fp8": fp8}


def _node_counts(case):
    """Nodes of each sequence's tree: given by the case alone."""
    return np.random.default_rng(case["lens"]).integers(case["n_lo"], case["n_hi"] + 1, size=case["batch"])


def _kv_lens(case):
    """Keys of each sequence, its nodes among them."""
    n = _node_counts(case)
    rng = np.random.default_rng(case["lens"] + 1)
    if case["kind"] == "tree":
        return np.maximum(n, rng.integers(case["lo"], case["hi"] + 1, size=case["batch"]))
    return n + rng.integers(0, case["block"] - 1, size=case["batch"])


def _trees(n, rng):
    """Ancestors [batch, N, N] (bool, self included) and parents [batch, N] of trees of n[b] nodes."""
    batch, most = n.size, int(n.max(initial=0))
    sees = np.zeros((batch, most, most), bool)
    parents = np.full((batch, most), -1)
    at = np.arange(batch)
    for i in range(most):
        if i:
            parents[:, i] = i - 1 - (rng.random(batch) ** 1.5 * min(i, 12)).astype(np.int64)     # mostly the last few nodes
            sees[:, i] = sees[at, parents[:, i]]
        sees[:, i, i] = True
    sees &= (np.arange(most) < n[:, None])[:, :, None]
    return sees, parents


def _words(sees, n):
    """One row of 64-bit words per node, packed node after node."""
    batch, most, _ = sees.shape
    words = max(1, -(-most // 64))
    bits = np.zeros((batch, most, words * 64), np.uint8)
    bits[:, :, :most] = sees
    packed = np.packbits(bits, axis=-1, bitorder="little").view(np.uint64).astype(np.uint64).view(np.int64)
    keep = np.arange(most) < n[:, None]
    return np.ascontiguousarray(packed[keep].reshape(-1, words))


def _paths(n, parents, sees, limit, rng):
    """An accepted path of each tree: to a random node, cut at `limit` nodes.  [batch, limit] padded with -1, lengths."""
    batch = n.size
    path = np.full((batch, limit), -1, np.int32)
    lens = np.zeros(batch, np.int32)
    for b in range(batch):
        if n[b]:
            nodes = np.flatnonzero(sees[b, rng.integers(0, n[b])])[:limit]
            path[b, :nodes.size] = nodes
            lens[b] = nodes.size
    return path, lens


def _fixed_paths(case):
    """Compaction moves as many rows as the case alone says."""
    n = _node_counts(case)
    rng = np.random.default_rng(case["lens"] + 2)
    sees, parents = _trees(n, rng)
    return _paths(n, parents, sees, case["path"], rng)


def _fixed_rows(case):
    return np.random.default_rng(case["lens"]).integers(case["r_lo"], case["r_hi"] + 1, size=case["pairs"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device=DEV, dtype=dtype)


def _running(n):
    return _dev(np.concatenate([[0], np.cumsum(n)]))


def _codes(shape, g):
    """e4m3 codes of every value but NaN."""
    c = torch.randint(0, 254, shape, generator=g, device=DEV, dtype=torch.uint8)
    c += (c >= 127).to(torch.uint8)
    return c.view(torch.float8_e4m3fn)


def _tables(kv_lens, block, rng, spare=1):
    """Block tables over a pool a quarter larger than the batch needs, blocks in random order; -1 past the end."""
    need = -(-kv_lens // block)
    total = int(need.sum()) + spare
    num_blocks = total + max(1, total // 4)
    table = np.full((kv_lens.size, max(1, int(need.max()))), -1, np.int32)
    ids = rng.permutation(num_blocks)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    return table, num_blocks


def _layer_pools(case, num_blocks, g):
    """All layers' pools in one allocation: [layers, 2 (K and V), num_blocks, block, hkv, D], and scales."""
    shape = (case["layers"], 2, num_blocks, case["block"], case["hkv"], D)
    if not case["fp8"]:
        return {"rows": torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16), "scales": None}
    scales = torch.randint(120, 128, shape[:3] + (case["hkv"], case["block"]), generator=g, device=DEV, dtype=torch.uint8)
    return {"rows": _codes(shape, g), "scales": scales.view(torch.float8_e8m0fnu)}


def prepare(case, seed):
    g = _gen(seed)
    rng = np.random.default_rng([int(seed), case["lens"]])
    s = {"kind": case["kind"]}
    if case["kind"] == "copy":
        rows = _fixed_rows(case)
        ids = rng.permutation(2 * case["pairs"] + 2)
        s.update(_layer_pools(case, ids.size, g))
        s.update(src=_dev(ids[:case["pairs"]]), dst=_dev(ids[case["pairs"]:2 * case["pairs"]]), count=_dev(rows))
        return s
    n = _node_counts(case)
    if case["kind"] == "compact":
        kl = _kv_lens(case)
        table, num_blocks = _tables(kl, case["block"], rng)
        path, lens = _fixed_paths(case)
        s.update(_layer_pools(case, num_blocks, g))
        s.update(tables=_dev(table), lens_k=_dev(kl), cu=_running(n), path=_dev(path), path_lens=_dev(lens))
        return s
    sees, parents = _trees(n, rng)
    s.update(cu=_running(n), mask=_dev(_words(sees, n), torch.int64), most=max(1, case["n_hi"]))
    if case["kind"] == "accept":
        # drafts from a small set of likely tokens (so that siblings may hold the same one), and at each
        # node the token sampled there: mostly one of its children's drafts
        batch, most = n.size, sees.shape[1]
        draft = rng.integers(0, 151936, size=(batch, most))
        twin = rng.random((batch, most)) < 0.1
        draft[:, 1:] = np.where(twin[:, 1:], draft[:, :-1], draft[:, 1:]) if most else draft[:, 1:]
        target = rng.integers(0, 151936, size=(batch, most))
        at = np.arange(batch)
        for i in range(1, most):
            take = (rng.random(batch) < 0.5) & (i < n)
            target[at[take], parents[take, i]] = draft[take, i]
        keep = np.arange(most) < n[:, None]
        s.update(draft=_dev(draft[keep], torch.int64), target=_dev(target[keep], torch.int64), path_most=case["path"],
                 lens_k=_dev(n + rng.integers(0, 4000, size=batch)))
        return s
    kl = _kv_lens(case)
    table, num_blocks = _tables(kl, case["block"], rng)
    shape = (num_blocks, case["block"], case["hkv"], D)
    if case["fp8"]:
        s.update(k_cache=_codes(shape, g), v_cache=_codes(shape, g))
        for name in ("k_scale", "v_scale"):
            # values of the codes have a root mean square of about 130
            s[name] = torch.randint(118, 122, (num_blocks, case["hkv"], case["block"]), generator=g, device=DEV, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    else:
        for name in ("k_cache", "v_cache"):
            s[name] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    q = torch.randn((int(n.sum()), case["hq"], D), generator=g, device=DEV, dtype=torch.bfloat16)
    s.update(q=q, out=torch.zeros_like(q), tables=_dev(table), lens_k=_dev(kl), max_k=int(kl.max()), scale=D ** -0.5,
             batch=case["batch"], hq=case["hq"], hkv=case["hkv"], fp8=case["fp8"])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _node_index(s):
    """[batch, N]: each tree's nodes in the packed order, and which of them exist."""
    n = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(s["most"], device=DEV)
    exists = i < n[:, None]
    at = torch.where(exists, s["cu"][:-1, None] + i, 0).long()
    return n, at, exists


def _sees(s, at, exists):
    """[batch, N, N] (bool) from the nodes' bits."""
    j = torch.arange(s["most"], device=DEV)
    if s["mask"].shape[0] == 0:
        return torch.zeros(at.shape + (s["most"],), dtype=torch.bool, device=DEV)
    bits = (s["mask"][:, j >> 6] >> (j & 63)) & 1
    return bits.bool()[at] & exists[:, :, None]


def _tree(s):
    n, at, exists = _node_index(s)
    block, hkv = s["k_cache"].shape[1], s["hkv"]
    batch, nodes, group = at.shape[0], at.shape[1], s["hq"] // hkv
    pos = torch.arange(s["max_k"], device=DEV)
    lens = s["lens_k"][:, None]
    phys = s["tables"].long()[:, pos // block]                                   # [B, L]
    valid = pos < lens
    slot = torch.where(valid, phys * block + pos % block, 0)

    def rows(name):
        if not s["fp8"]:
            return s[name + "_cache"].view(-1, hkv, D)[slot].float()
        value = s[name + "_cache"].view(torch.uint8).view(-1, hkv, D)[slot].view(torch.float8_e4m3fn).float()
        byte = s[name + "_scale"].view(torch.uint8).permute(0, 2, 1).reshape(-1, hkv)[slot]
        return value * torch.exp2(byte.float() - 127.0).unsqueeze(-1)

    q = s["q"][at].float().view(batch, nodes, hkv, group, D).permute(0, 2, 1, 3, 4).reshape(batch, hkv, nodes * group, D)
    scores = torch.matmul(q, rows("k").permute(0, 2, 3, 1)) * s["scale"]         # [B, hkv, N G, L]
    first = (s["lens_k"] - n)[:, None]
    node = (pos - first).clamp(0, nodes - 1)                                     # [B, L]
    shown = torch.gather(_sees(s, at, exists), 2, node[:, None, :].expand(batch, nodes, pos.numel()))
    shown = (shown | (pos < first)[:, None, :]) & valid[:, None, :]
    shown = shown.repeat_interleave(group, 1)[:, None]                           # [B, 1, N G, L]
    scores = torch.where(shown, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    w = torch.exp(scores - torch.where(top > -math.inf, top, 0.0))
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-38)
    out = torch.matmul(w, rows("v").permute(0, 2, 1, 3))                         # [B, hkv, N G, D]
    out = out.view(batch, hkv, nodes, group, D).permute(0, 2, 1, 3, 4).reshape(batch, nodes, s["hq"], D)
    return out[exists].to(torch.bfloat16)


def _accept(s):
    n, at, exists = _node_index(s)
    i = torch.arange(s["most"], device=DEV)
    limit = s["path_most"]
    if s["draft"].shape[0] == 0:
        return {"path": torch.full((n.shape[0], limit), -1, dtype=torch.int32, device=DEV), "lens": torch.zeros_like(n), "next": torch.full_like(n, -1, dtype=torch.int64),
                "context": s["lens_k"].clone()}
    above = _sees(s, at, exists) & (i < i[:, None])                              # ancestors
    parent = torch.where(above, i, -1).amax(-1)                                  # [B, N]
    draft, target = s["draft"][at], s["target"][at]
    hit = (parent >= 0) & exists & (draft == torch.gather(target, 1, parent.clamp(min=0)))
    twin = (parent[:, :, None] == parent[:, None, :]) & (draft[:, :, None] == draft[:, None, :]) & hit[:, None, :] & (i < i[:, None])
    good = (hit & ~twin.any(-1)) | ((i == 0) & exists)
    taken = good & ~(above & ~good[:, None, :]).any(-1)
    depth = torch.cumsum(taken.int(), 1) - 1
    taken &= depth < limit
    lens = taken.sum(1).int()
    path = torch.full((n.shape[0], limit + 1), -1, dtype=torch.int32, device=DEV)
    path.scatter_(1, torch.where(taken, depth, limit).long(), i.int().expand_as(taken).contiguous())
    last = torch.where(taken, i, -1).amax(1)
    follow = torch.where(last >= 0, torch.gather(target, 1, last.clamp(min=0)[:, None])[:, 0], -1)
    return {"path": path[:, :limit].contiguous(), "lens": lens, "next": follow, "context": s["lens_k"] - n + lens}


def _move(s, src_block, src_row, dst_block, dst_row):
    """Rows (and their scales) of every layer copied; all are read before any is written."""
    if s["scales"] is None:
        s["rows"][:, :, dst_block, dst_row] = s["rows"][:, :, src_block, src_row]
        return {"rows": s["rows"]}
    rows, scales = s["rows"].view(torch.uint8), s["scales"].view(torch.uint8)
    rows[:, :, dst_block, dst_row] = rows[:, :, src_block, src_row]
    scales[:, :, dst_block, :, dst_row] = scales[:, :, src_block, :, src_row]
    return {"rows": s["rows"], "scales": s["scales"]}


def _compact(s):
    block = s["rows"].shape[3]
    depth = torch.arange(s["path"].shape[1], device=DEV)
    first = (s["lens_k"] - (s["cu"][1:] - s["cu"][:-1]))[:, None]
    moved = (depth < s["path_lens"][:, None]) & (s["path"] != depth)
    seq = torch.arange(first.shape[0], device=DEV)[:, None].expand_as(moved)[moved]
    src, dst = (first + s["path"])[moved].long(), (first + depth)[moved].long()
    table = s["tables"].long()
    return _move(s, table[seq, src // block], src % block, table[seq, dst // block], dst % block)


def _copy(s):
    row = torch.arange(s["rows"].shape[3], device=DEV)
    kept = row < s["count"][:, None]
    src, dst, row = (t.expand_as(kept)[kept].long() for t in (s["src"][:, None], s["dst"][:, None], row))
    return _move(s, src, row, dst, row)


def _pools(pkv, s):
    """The handle that a serving program makes once for all its layers' pools."""
    if "pools" not in s:
        k, v = s["rows"].unbind(1)
        scales = () if s["scales"] is None else tuple(list(t) for t in s["scales"].unbind(1))
        s["pools"] = pkv.KvPools(list(k), list(v), *scales)
    return s["pools"]


def run(state):
    s = state
    if own:
        import paged_kv_attention_29_gb300 as pkv
        if s["kind"] == "tree":
            if "workspace" not in s:     # a serving program keeps it for every step
                s["workspace"] = pkv.tree_decode_workspace(s["batch"], s["most"], s["hq"], s["hkv"], D)
            if s["fp8"]:
                return pkv.pkv_tree_decode_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["tables"], s["lens_k"], s["cu"],
                                               s["mask"], s["most"], s["max_k"], s["scale"], out=s["out"], workspace=s["workspace"])
            return pkv.pkv_tree_decode(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens_k"], s["cu"], s["mask"], s["most"], s["max_k"],
                                       s["scale"], out=s["out"], workspace=s["workspace"])
        if s["kind"] == "accept":
            path, lens, follow, context = pkv.pkv_tree_accept(s["target"], s["draft"], s["mask"], s["cu"], s["lens_k"], s["most"], s["path_most"])
            return {"path": path, "lens": lens, "next": follow, "context": context}
        pools = _pools(pkv, s)
        if s["kind"] == "compact":
            pkv.pkv_tree_compact(pools, s["tables"], s["lens_k"], s["cu"], s["path"], s["path_lens"])
        else:
            pkv.pkv_copy_blocks(pools, s["src"], s["dst"], s["count"])
        return {"rows": s["rows"]} if s["scales"] is None else {"rows": s["rows"], "scales": s["scales"]}
    return {"tree": _tree, "accept": _accept, "compact": _compact, "copy": _copy}[s["kind"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["kind"] == "tree":
        n, kl = _node_counts(case), _kv_lens(case)
        row = 2 * case["hkv"] * ((D + 1) if case["fp8"] else 2 * D)
        words = -(-case["n_hi"] // 64)
        return {"bytes": int(kl.sum()) * row + int(n.sum()) * (case["hq"] * D * 4 + 8 * words), "flops": 4 * D * case["hq"] * int((n * kl).sum())}
    if case["kind"] == "accept":
        n = _node_counts(case)
        words = max(1, -(-int(n.max()) // 64))
        return {"bytes": int(n.sum()) * (8 * words + 16) + case["batch"] * (4 * case["path"] + 24), "flops": 0}
    row = case["layers"] * 2 * case["hkv"] * ((D + 1) if case["fp8"] else 2 * D)
    if case["kind"] == "compact":
        path, lens = _fixed_paths(case)
        depth = np.arange(case["path"])
        moved = int(((depth < lens[:, None]) & (path != depth)).sum())
        return {"bytes": max(1, 2 * moved * row), "flops": 0}
    return {"bytes": max(1, 2 * int(_fixed_rows(case).sum()) * row), "flops": 0}


def exact(case, seed):
    if case["kind"] != "tree":
        return None                  # whole numbers, and rows that are only moved
    s = prepare(case, seed)
    block, hkv, group = case["block"], case["hkv"], case["hq"] // case["hkv"]
    tables, lens, cu = s["tables"].cpu().numpy(), s["lens_k"].cpu().numpy(), s["cu"].cpu().numpy()
    words = s["mask"].cpu().numpy().view(np.uint64)
    got = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(case["batch"]):
        lo, hi, keys = int(cu[b]), int(cu[b + 1]), int(lens[b])
        n = hi - lo
        blocks = torch.from_numpy(tables[b, :-(-keys // block)].astype(np.int64)).to(DEV)
        seen = torch.ones((n, keys), dtype=torch.bool)
        for i in range(n):
            seen[i, keys - n:] = torch.tensor([bool(int(words[lo + i, j // 64]) >> (j % 64) & 1) for j in range(n)])
        seen = seen.to(DEV)
        for h in range(hkv):
            k, v = (s[x + "_cache"][blocks, :, h].reshape(-1, D)[:keys].double() if not case["fp8"] else
                    s[x + "_cache"].view(torch.uint8)[blocks, :, h].view(torch.float8_e4m3fn).reshape(-1, D)[:keys].double()
                    * s[x + "_scale"].view(torch.uint8)[blocks, h].view(torch.float8_e8m0fnu).reshape(-1)[:keys, None].double() for x in "kv")
            for e in range(group):
                z = (s["q"][lo:hi, h * group + e].double() @ k.T) * s["scale"]
                z = z.masked_fill(~seen, -math.inf)
                got[lo:hi, h * group + e] = torch.nan_to_num(torch.softmax(z, -1)) @ v
    return got
