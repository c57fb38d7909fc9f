"""The serving operators on an 8-bit KV cache, and filtered sampling: cases, inputs and plain forms.

An 8-bit cache holds every K/V row (one token, one KV head, 128 numbers) as 128
e4m3 codes and one power-of-two scale (E8M0: byte b stands for 2^(b - 127)):

  append    (rotate q and k by their positions,) round the K/V rows to e4m3 with a scale
            each and write them to their pool slots
  decode    attention of one new token per sequence over that cache
  prefill   causal attention of packed prompts over that cache
  sample    one token per row of logits by temperature, top-k, top-p and min-p

`own` chooses between the plain forms here (elementary torch operations) and the
library's kernels.
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
ROPE_BASE = 1.0e6
SHAPES = ((16, 8), (16, 16), (16, 4), (32, 4), (8, 1))     # query heads, KV heads


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one sequence's new token, as each layer of a single-stream decode step appends it: latency
        {"name": "append one token", "kind": "append", "n": 1, "hq": 16, "hkv": 8, "block": 256, "rope": True, "pad": False},
        # an odd batch padded to a captured graph's size (skipped rows), K already rotated by the model
        {"name": "append padded, no rotation", "kind": "append", "n": 259, "hq": 32, "hkv": 4, "block": 512, "rope": False, "pad": True},
        # the new tokens of 32 prompts of 100 to 1024 tokens after their prefix hits
        {"name": "append a prefill batch", "kind": "append", "n": 10814, "hq": 16, "hkv": 8, "block": 256, "rope": True, "pad": False},
        # a single short conversation: latency
        {"name": "decode one sequence", "kind": "decode", "batch": 1, "lo": 301, "hi": 301, "lens": 1, "hq": 16, "hkv": 8, "block": 256},
        # a serving batch, 512 to 4096 tokens of context
        {"name": "decode batch of 64", "kind": "decode", "batch": 64, "lo": 512, "hi": 4096, "lens": 2, "hq": 16, "hkv": 8, "block": 256},
        # long documents: few sequences, so each is split over its length
        {"name": "decode long contexts", "kind": "decode", "batch": 8, "lo": 16384, "hi": 40960, "lens": 3, "hq": 16, "hkv": 8, "block": 256},
        # eight query heads to a KV head, uneven lengths, finished sequences (length 0) left in the batch
        {"name": "decode wide groups, ragged", "kind": "decode", "batch": 37, "lo": 0, "hi": 2999, "lens": 4, "hq": 32, "hkv": 4, "block": 512},
        # a short follow-up question on a cached conversation: latency
        {"name": "prefill a follow-up", "kind": "prefill", "batch": 1, "lo": 293, "hi": 293, "cached": 0.87, "lens": 5, "hq": 16, "hkv": 8, "block": 256},
        # 32 prompts of 100 to 1024 tokens, part of each cached by a shared prefix
        {"name": "prefill 32 prompts", "kind": "prefill", "batch": 32, "lo": 100, "hi": 1024, "cached": 0.5, "lens": 6, "hq": 16, "hkv": 8, "block": 256},
        # one long document, nothing cached
        {"name": "prefill a long prompt", "kind": "prefill", "batch": 1, "lo": 8192, "hi": 8192, "cached": 0.0, "lens": 7, "hq": 16, "hkv": 8, "block": 256},
        # one request's next token: latency
        {"name": "sample one row", "kind": "sample", "batch": 1, "vocab": 151936, "std": 3.0, "rounded": True, "masked": 0.0, "rows": 8},
        # a full decode batch, every request with settings of its own
        {"name": "sample 256 rows", "kind": "sample", "batch": 256, "vocab": 151936, "std": 3.0, "rounded": False, "masked": 0.0, "rows": 9},
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(("append", "decode", "prefill", "sample"))
    hq, hkv = rng.choice(SHAPES)
    block = rng.choice((256, 256, 512))
    lens = rng.randrange(1 << 30)
    if kind == "append":
        return {"kind": kind, "n": _log_int(rng, 1, 10000), "hq": hq, "hkv": hkv, "block": block,
                "rope": rng.random() < 0.7, "pad": rng.random() < 0.4}
    if kind == "decode":
        batch = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, min(40960, 260000 // batch))
        return {"kind": kind, "batch": batch, "lo": rng.randint(0 if batch > 4 else 1, hi), "hi": hi, "lens": lens, "hq": hq, "hkv": hkv, "block": block}
    if kind == "prefill":
        batch = _log_int(rng, 1, 32)
        hi = _log_int(rng, 2, int(8000 / math.sqrt(batch)))
        return {"kind": kind, "batch": batch, "lo": rng.randint(1, hi), "hi": hi, "cached": rng.choice((0.0, 0.3, 0.9)),
                "lens": lens, "hq": min(hq, 16), "hkv": hkv, "block": block}
    batch = _log_int(rng, 1, 256)
    return {"kind": kind, "batch": batch, "vocab": _log_int(rng, 100, 151936), "std": rng.choice((0.5, 1.5, 3.0, 5.0)),
            "rounded": rng.random() < 0.5, "masked": rng.choice((0.0, 0.0, 0.7)), "rows": lens}


def _kv_lens(case):
    """Keys of each sequence: given by the case alone."""
    return np.random.default_rng(case["lens"]).integers(case["lo"], case["hi"] + 1, size=case["batch"])


def _q_lens(case):
    """New tokens of each prompt: what its cached share leaves, at least one."""
    kl = _kv_lens(case)
    share = np.random.default_rng(case["lens"] + 1).uniform(0.0, 2.0 * case["cached"], size=case["batch"])
    share = np.full_like(share, case["cached"]) if case["batch"] == 1 else np.minimum(share, 1.0)
    return np.maximum(1, kl - (kl * share).astype(np.int64))


def _row_settings(case):
    """Each row's temperature, top-k, top-p and min-p, as requests set them (0, 1 and 0: off)."""
    rng = np.random.default_rng(case["rows"])
    n = case["batch"]
    return (rng.uniform(0.5, 1.2, n).astype(np.float32),
            rng.choice(np.array([0, 0, 1, 5, 20, 50, 200, 1000], np.int32), n),
            np.where(rng.random(n) < 0.3, 1.0, rng.uniform(0.5, 1.0, n)).astype(np.float32),
            np.where(rng.random(n) < 0.6, 0.0, rng.uniform(0.005, 0.2, n)).astype(np.float32))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _pool(shape, g):
    """A filled pool: rows of normal values whose size differs from row to row, in 8 bits.
    Returns codes [num_blocks, block, hkv, D] and scales [num_blocks, hkv, block]."""
    x = _randn(shape, g)
    x *= torch.exp2(torch.randint(-2, 2, shape[:3], generator=g, device=DEV).float()).unsqueeze(-1) * 0.8
    codes, scale = _to_8_bits(x)
    return codes, scale.permute(0, 2, 1).contiguous()


def _tables(kv_lens, block, rng):
    """Block tables over a pool a quarter larger than the batch needs, blocks in random order; -1 past the end."""
    need = -(-kv_lens // block)
    total = int(need.sum()) + 1
    num_blocks = total + total // 4
    perm = rng.permutation(num_blocks).astype(np.int32)
    width = max(1, int(need.max()))
    col = np.arange(width)[None, :]
    first = (np.cumsum(need) - need)[:, None]
    return num_blocks, np.where(col < need[:, None], perm[np.minimum(first + col, num_blocks - 1)], -1).astype(np.int32)


def prepare(case, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    s = dict(case)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    if case["kind"] == "sample":
        t, k, p, m = _row_settings(case)
        logits = _randn((case["batch"], case["vocab"]), g) * case["std"]
        if case["rounded"]:          # logits of a bf16 output projection: many equal values
            logits = logits.bfloat16().float()
        if case["masked"]:           # a grammar's mask
            out = torch.rand(logits.shape, generator=g, device=DEV) < case["masked"]
            out[:, int(rng.integers(0, case["vocab"]))] = False
            logits = logits.masked_fill(out, -math.inf)
        s.update(logits=logits, t=dev(t), top_k=dev(k), top_p=dev(p), min_p=dev(m), seed=int(rng.integers(0, 1 << 62)),
                 offset=int(rng.integers(0, 1 << 20)), ids=torch.empty(case["batch"], dtype=torch.int64, device=DEV))
        return s
    hq, hkv, block = case["hq"], case["hkv"], case["block"]
    if case["kind"] == "append":
        n = case["n"]
        qkv = _randn((n, hq + 2 * hkv, D), g)
        qkv[:, hq:] *= torch.exp2(torch.randint(-3, 4, (n, 2 * hkv, 1), generator=g, device=DEV).float())
        qkv = qkv.bfloat16()         # one fused projection's output: q, k and v are views into it
        blocks = -(-n // block)
        num_blocks = blocks + blocks // 4 + 1
        perm = rng.permutation(num_blocks)
        at = np.arange(n)
        slots = perm[at // block] * block + at % block
        if case["pad"]:
            slots = np.where(at % 7 == 3, -1, slots)
        k_cache, k_scale = _pool((num_blocks, block, hkv, D), g)
        v_cache, v_scale = _pool((num_blocks, block, hkv, D), g)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], positions=dev(rng.integers(0, 131072, n).astype(np.int32)),
                 slots=dev(slots.astype(np.int32)), k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                 q_out=torch.empty((n, hq, D), dtype=torch.bfloat16, device=DEV))
        return s
    kl = _kv_lens(case)
    num_blocks, tables = _tables(kl, block, rng)
    k_cache, k_scale = _pool((num_blocks, block, hkv, D), g)
    v_cache, v_scale = _pool((num_blocks, block, hkv, D), g)
    s.update(k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, tables=dev(tables), scale=D ** -0.5,
             max_k=max(1, int(kl.max())))
    if case["kind"] == "decode":
        q = (1.5 * _randn((case["batch"], hq, D), g)).bfloat16()
        s.update(q=q, lens_k=dev(kl.astype(np.int32)), out=torch.empty_like(q))
        return s
    ql = _q_lens(case)
    run_on = lambda a: np.concatenate([[0], np.cumsum(a)]).astype(np.int32)  # noqa: E731
    q = (1.5 * _randn((int(ql.sum()), hq, D), g)).bfloat16()
    s.update(q=q, cu_q=dev(run_on(ql)), cu_k=dev(run_on(kl)), max_q=int(ql.max()), total_k=int(kl.sum()), out=torch.empty_like(q))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _to_8_bits(x):
    """Rows of fp32 (last axis) as e4m3 codes and one E8M0 scale each: the smallest power of two, at least
    2^-126, under which the row's largest magnitude is at most 448.  A row with an infinity or a NaN gets the
    scale NaN and codes 0."""
    amax = x.abs().amax(-1)
    whole = torch.isfinite(amax)
    m, e = torch.frexp(torch.where(whole, amax, 1.0))             # amax = m 2^e, 1/2 <= m < 1
    e = torch.where(m <= 0.875, e - 9, e - 8)                     # 448 = 0.875 2^9
    e = torch.where(amax == 0, -126, e).clamp(min=-126)
    scaled = torch.where(whole.unsqueeze(-1), x * torch.exp2(-e.float()).unsqueeze(-1), 0.0)
    byte = torch.where(whole, e + 127, 255).to(torch.uint8)
    return scaled.to(torch.float8_e4m3fn), byte.view(torch.float8_e8m0fnu)


def _turned(x, cos, sin):
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append(s):
    k, v = s["k"].float(), s["v"].float()
    q_out = None
    if s["rope"]:
        freq = ROPE_BASE ** (-2.0 * torch.arange(D // 2, device=k.device, dtype=torch.float64) / D)
        angle = s["positions"].double()[:, None] * freq           # 64 bits: angles of far positions
        cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
        k = _turned(k, cos, sin)
        q_out = _turned(s["q"].float(), cos, sin).bfloat16()
    block = s["block"]
    slots = s["slots"].long()
    valid = slots >= 0
    row = torch.where(valid, torch.arange(len(slots), device=slots.device), valid.int().argmax())   # a skipped row repeats a written one
    slot = slots[row]
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
        codes, e = _to_8_bits(x)
        cache.view(torch.uint8)[slot // block, slot % block] = codes.view(torch.uint8)[row]
        scale.view(torch.uint8)[slot // block, :, slot % block] = e.view(torch.uint8)[row]
    return _appended(s, q_out)


def _appended(s, q_out):
    out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if q_out is not None:
        out["q_out"] = q_out
    return out


def _gathered(cache, scale, tables, n, block):
    """The first n keys' rows of each sequence as fp32 [batch, hkv, n, D]."""
    at = torch.arange(n, device=tables.device)
    blk = tables[:, at // block].clamp(min=0).long()
    off = (at % block)[None, :].expand_as(blk)
    codes = cache.view(torch.uint8)[blk, off].view(torch.float8_e4m3fn).float()
    sc = scale.view(torch.uint8)[blk, :, off].view(torch.float8_e8m0fnu).float()
    return (codes * sc.unsqueeze(-1)).permute(0, 2, 1, 3)


def _softmaxed(scores, seen):
    """Softmax over the last axis of what `seen` leaves; rows that see nothing are 0."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total)


def _decode(s):
    q, hkv = s["q"].float(), s["hkv"]
    k = _gathered(s["k_cache"], s["k_scale"], s["tables"], s["max_k"], s["block"])
    v = _gathered(s["v_cache"], s["v_scale"], s["tables"], s["max_k"], s["block"])
    scores = torch.matmul(q.view(len(q), hkv, -1, D) * s["scale"], k.transpose(-1, -2))
    seen = torch.arange(s["max_k"], device=q.device) < s["lens_k"][:, None, None, None]
    return torch.matmul(_softmaxed(scores, seen), v).reshape(q.shape).bfloat16()


def _prefill(s):
    q, hkv, cu_q, cu_k = s["q"], s["hkv"], s["cu_q"].long(), s["cu_k"].long()
    ql, kl = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i = torch.arange(s["max_q"], device=q.device)
    rows = (cu_q[:-1, None] + torch.minimum(i, (ql - 1)[:, None])).clamp(min=0)
    qp = q[rows].float().view(len(ql), s["max_q"], hkv, -1, D).permute(0, 2, 3, 1, 4)        # [batch, hkv, G, max_q, D]
    k = _gathered(s["k_cache"], s["k_scale"], s["tables"], s["max_k"], s["block"])
    v = _gathered(s["v_cache"], s["v_scale"], s["tables"], s["max_k"], s["block"])
    scores = torch.matmul(qp * s["scale"], k.transpose(-1, -2).unsqueeze(2))
    j = torch.arange(s["max_k"], device=q.device)
    last = (i[None, :] + (kl - ql)[:, None]).clamp(max=kl.max())
    seen = (j <= last[:, :, None]) & (j < kl[:, None, None])
    o = torch.matmul(_softmaxed(scores, seen[:, None, None]), v.unsqueeze(2)).permute(0, 3, 1, 2, 4)
    t = torch.arange(len(q), device=q.device)
    seq = torch.searchsorted(cu_q[1:].contiguous(), t, right=True)
    return o[seq, t - cu_q[seq]].reshape(q.shape).bfloat16()


_LOW = 0xFFFFFFFF


def _round(c, key):
    """One Philox4x32 round on counters of 32-bit words held in 64 bits."""
    p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
    return ((p1 >> 32) & _LOW) ^ c[1] ^ key[0], p1 & _LOW, ((p0 >> 32) & _LOW) ^ c[3] ^ key[1], p0 & _LOW


def _uniforms(seed, offset, rows, vocab, dev):
    """The noise of every (row, column): Philox4x32-10 with key `seed` and counter (column // 4, row + offset, 0), word
    column % 4 as an odd multiple of 2^-24."""
    quads = -(-vocab // 4)
    r = torch.arange(rows, device=dev, dtype=torch.int64)[:, None].expand(rows, quads) + offset
    q = torch.arange(quads, device=dev, dtype=torch.int64)[None, :].expand(rows, quads)
    c = (q, r & _LOW, (r >> 32) & _LOW, torch.zeros_like(q))
    keys = [((seed + n * 0x9E3779B9) & _LOW, ((seed >> 32) + n * 0xBB67AE85) & _LOW) for n in range(10)]
    c = _round(_round(_round(_round(_round(c, keys[0]), keys[1]), keys[2]), keys[3]), keys[4])
    c = _round(_round(_round(_round(_round(c, keys[5]), keys[6]), keys[7]), keys[8]), keys[9])
    x = torch.stack(c, -1).view(rows, quads * 4)[:, :vocab]
    return (2 * (x >> 9) + 1).double() * 2.0 ** -24


def _sample(s):
    logits, dev = s["logits"], s["logits"].device
    rows, vocab = logits.shape
    ranked, order = torch.sort(logits, dim=1, descending=True, stable=True)        # equal logits: lowest column first
    z = (ranked.double() - ranked[:, :1].double()) / s["t"].double()[:, None]      # 64 bits: sums next to a border
    rank = torch.arange(vocab, device=dev)
    k = s["top_k"][:, None]
    kept = (ranked > -math.inf) & ((k <= 0) | (rank < k))
    w = torch.exp(z) * kept
    before = torch.cumsum(w, 1) - w
    p = s["top_p"].double()[:, None]
    kept &= (p >= 1) | (before < p * w.sum(1, keepdim=True))
    kept &= z >= torch.log(s["min_p"].double())[:, None]
    u = _uniforms(s["seed"], s["offset"], rows, vocab, dev).gather(1, order)
    key = torch.where(kept, z - torch.log(-torch.log(u)), -math.inf)
    best = key.amax(1, keepdim=True)
    return torch.where(key == best, order, vocab).amin(1)


def run(state):
    s = state
    if own:
        import paged_kv_attention_29_gb300 as pkv
        if s["kind"] == "append":
            pools = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
            if s["rope"]:
                return _appended(s, pkv.pkv_rope_store_kvcache_fp8(s["q"], s["k"], s["v"], s["positions"], s["slots"], *pools, ROPE_BASE, q_out=s["q_out"]))
            pkv.pkv_store_kvcache_fp8(s["k"], s["v"], s["slots"], *pools)
            return _appended(s, None)
        if s["kind"] == "decode":
            if "workspace" not in s:     # a serving program keeps it for every step
                s["workspace"] = pkv.decode_fp8_workspace(s["batch"], s["hq"], s["hkv"], D)
            return pkv.pkv_decode_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["tables"], s["lens_k"], s["max_k"],
                                      s["scale"], out=s["out"], workspace=s["workspace"])
        if s["kind"] == "prefill":
            if "workspace" not in s:
                s["workspace"] = pkv.prefill_fp8_workspace(s["batch"], s["hq"], s["hkv"], D, s["max_q"], s["max_k"], s["total_k"])
            return pkv.pkv_prefill_varlen_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["cu_q"], s["cu_k"], s["tables"],
                                              s["max_q"], s["max_k"], s["total_k"], s["scale"], out=s["out"], workspace=s["workspace"])
        return pkv.pkv_sample_filtered(s["logits"], s["t"], s["top_k"], s["top_p"], s["min_p"], s["seed"], s["offset"], out_ids=s["ids"])
    return {"append": _append, "decode": _decode, "prefill": _prefill, "sample": _sample}[s["kind"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["kind"] == "sample":
        return {"bytes": case["batch"] * (case["vocab"] * 4 + 4 * 4 + 8), "flops": 4 * case["batch"] * case["vocab"]}
    hq, hkv = case["hq"], case["hkv"]
    if case["kind"] == "append":
        at = np.arange(case["n"])
        written = int((at % 7 != 3).sum()) if case["pad"] else case["n"]
        turned = case["n"] * (hq * 4 * D + 4) if case["rope"] else 0
        return {"bytes": written * 2 * hkv * (2 * D + D + 1) + case["n"] * 4 + turned, "flops": 4 * written * 2 * hkv * D}
    kl = _kv_lens(case)
    row = 2 * hkv * (D + 1)
    if case["kind"] == "decode":
        return {"bytes": int(kl.sum()) * row + case["batch"] * hq * D * 4, "flops": 4 * D * hq * int(kl.sum())}
    ql = _q_lens(case)
    pairs = int((ql * kl - ql * (ql - 1) // 2).sum())
    return {"bytes": int(kl.sum()) * row + int(ql.sum()) * hq * D * 4, "flops": 4 * D * hq * pairs}


def _exact_8_bits(x):
    """x: float64 [..., D].  The codes' values and the scales' values, from the formats' definitions."""
    amax = np.abs(x).max(-1)
    e = np.ceil(np.log2(np.maximum(amax, 2.0 ** -140) / 448.0))
    e = np.where(amax <= 448.0 * 2.0 ** (e - 1), e - 1, np.where(amax > 448.0 * 2.0 ** e, e + 1, e))
    e = np.maximum(e, -126)
    y = x / 2.0 ** e[..., None]
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -20))), -6) - 3)     # 3 bits behind the point, subnormal below 2^-6
    return np.rint(y / step) * step, 2.0 ** e


def exact(case, seed):
    if case["kind"] == "sample":
        return None                  # whole numbers only
    s = prepare(case, seed)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    if case["kind"] == "append":
        k, v, pos = host(s["k"]), host(s["v"]), host(s["positions"])
        z = np.exp(1j * pos[:, None] * ROPE_BASE ** (-np.arange(D // 2) / (D // 2)))[:, None, :]
        spin = lambda x: (lambda w: np.concatenate([w.real, w.imag], -1))((x[..., :D // 2] + 1j * x[..., D // 2:]) * z)  # noqa: E731
        slots = s["slots"].cpu().numpy()
        got = {n: host(s[n]) for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
        for name, x in (("k", spin(k) if case["rope"] else k), ("v", v)):
            y, e = _exact_8_bits(x)
            keep = slots >= 0
            blk, off = slots[keep] // case["block"], slots[keep] % case["block"]
            got[name + "_cache"][blk, off] = y[keep]
            got[name + "_scale"][blk, :, off] = e[keep]
        if case["rope"]:
            got["q_out"] = spin(host(s["q"]))
        return got
    group = case["hq"] // case["hkv"]
    k8, v8 = s["k_cache"], s["v_cache"]
    ks, vs = s["k_scale"], s["v_scale"]
    kl = _kv_lens(case)
    ql = _q_lens(case) if case["kind"] == "prefill" else np.ones_like(kl)
    q = s["q"].double()
    out = torch.zeros_like(q)
    row = 0
    for b in range(case["batch"]):
        n, m = int(kl[b]), int(ql[b])
        blocks = s["tables"][b, :-(-n // case["block"])].long()
        for h in range(case["hkv"]):
            if n == 0:
                continue
            kh = (k8[blocks, :, h].double() * ks[blocks, h].double()[..., None]).reshape(-1, D)[:n]
            vh = (v8[blocks, :, h].double() * vs[blocks, h].double()[..., None]).reshape(-1, D)[:n]
            for g in range(h * group, (h + 1) * group):
                a = q[row:row + m, g] @ kh.T * s["scale"]
                if m > 1 or case["kind"] == "prefill":
                    a = a + torch.triu(torch.full_like(a, -math.inf), diagonal=n - m + 1)
                out[row:row + m, g] = torch.softmax(a, -1) @ vh
        row += m
    return out
