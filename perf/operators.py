"""Cases of the 4-bit KV cache's operators: append and read back, attention over the cache (causal, sliding window, first
tokens kept visible), accumulated attention weights, eviction by them.

Each case runs either in its plain form (elementary torch operations in 32 bits on the cache's own bytes) or, with `own`
set, through ``lossless_bf16_kv_amd.kv4``.  Both work on the same paged buffers:

    k_codes  uint8 [pages, kv_heads, page, D / 2]           two E2M1 codes a byte, the even channel in the low nibble
    k_scales uint8 [pages, kv_heads, page, D / 32]          2^(byte - 127) for each 32 channels
    v_codes  uint8 [pages, kv_heads, page / 4, 16, 4, D/32] four tokens interleaved, D / 16 channels of each at a time
    v_scales uint8 [pages, kv_heads, D / 32, page]
    weights  fp32  [pages, kv_heads, page]                  accumulated attention weight of each token

Token j of sequence s lies in page table[s, j // page] at j % page.  `lens` counts a sequence's tokens with the new ones;
its n = cu[s + 1] - cu[s] queries (or appended tokens) are its last n tokens.
"""
import math

import numpy as np
import torch

own = False

NIBBLE = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of 64 requests writes one token each: launch-bound
        {"name": "append-step", "op": "append", "dtype": "bf16", "hkv": 8, "d": 128, "page": 64, "seqs": 64, "lo": 100,
         "hi": 4096, "qlo": 1, "qhi": 1, "seed": 1},
        # the KV of one layer of a 32768-token prefill goes into the cache, K and V being slices of one projection
        {"name": "append-prefill", "op": "append", "dtype": "bf16", "hkv": 8, "d": 128, "page": 64, "seqs": 1, "lo": 32768,
         "hi": 32768, "qlo": 32768, "qhi": 32768, "seed": 2},
        # one chat request decoding: the smallest attention call
        {"name": "attend-one", "op": "attend", "dtype": "bf16", "hq": 64, "hkv": 8, "d": 128, "page": 64, "seqs": 1,
         "lo": 4097, "hi": 4097, "qlo": 1, "qhi": 1, "window": 0, "sinks": 0, "seed": 3},
        # a decode step of 256 requests of 128 to 8192 tokens
        {"name": "attend-ragged", "op": "attend", "dtype": "bf16", "hq": 64, "hkv": 8, "d": 128, "page": 64, "seqs": 256,
         "lo": 128, "hi": 8192, "qlo": 1, "qhi": 1, "window": 0, "sinks": 0, "seed": 7},
        # a decode step after long prefills
        {"name": "attend-long", "op": "attend", "dtype": "bf16", "hq": 64, "hkv": 8, "d": 128, "page": 64, "seqs": 32,
         "lo": 32768, "hi": 32768, "qlo": 1, "qhi": 1, "window": 0, "sinks": 0, "seed": 4},
        # the same caches read through a window with the first tokens kept, fp16 activations, small pages
        {"name": "attend-window", "op": "attend", "dtype": "fp16", "hq": 64, "hkv": 8, "d": 128, "page": 16, "seqs": 32,
         "lo": 20001, "hi": 32768, "qlo": 1, "qhi": 1, "window": 4096, "sinks": 4, "seed": 5},
        # checking drafted tokens: a few queries a request, narrow heads
        {"name": "attend-draft", "op": "attend", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 64, "page": 32, "seqs": 24,
         "lo": 1000, "hi": 8192, "qlo": 3, "qhi": 6, "window": 0, "sinks": 0, "seed": 6},
        # a prefill chunk of 4096 tokens on top of 4096 cached ones
        {"name": "attend-chunk", "op": "attend", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 64, "seqs": 1,
         "lo": 8192, "hi": 8192, "qlo": 4096, "qhi": 4096, "window": 0, "sinks": 0, "seed": 8},
        # weights of a decode step added up
        {"name": "weigh-step", "op": "weigh", "dtype": "bf16", "hq": 64, "hkv": 8, "d": 128, "page": 64, "seqs": 64,
         "lo": 128, "hi": 8192, "qlo": 1, "qhi": 1, "window": 0, "sinks": 0, "seed": 9},
        # weights of a prompt's last 1000 queries, read before the prompt's cache is cut down
        {"name": "weigh-prompt", "op": "weigh", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 64, "seqs": 2,
         "lo": 16000, "hi": 16384, "qlo": 1000, "qhi": 1000, "window": 0, "sinks": 0, "seed": 10},
        # 64 requests cut down to 2048 tokens a head
        {"name": "evict-ragged", "op": "evict", "hkv": 8, "d": 128, "page": 64, "seqs": 64, "lo": 128, "hi": 8192,
         "budget": 2048, "sinks": 4, "recent": 256, "seed": 11},
        # four long prefills cut down to an odd budget
        {"name": "evict-long", "op": "evict", "hkv": 8, "d": 128, "page": 64, "seqs": 4, "lo": 32768, "hi": 32768,
         "budget": 8191, "sinks": 16, "recent": 1024, "seed": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weigh", "evict"])
    c = {"op": op, "hkv": rng.choice([1, 2, 4, 8]), "d": rng.choice([64, 128, 128, 256]),
         "page": rng.choice([16, 32, 64, 128]), "seed": rng.randrange(1 << 20)}
    if op != "evict":
        c["dtype"] = rng.choice(["bf16", "bf16", "fp16"])
    seqs = _log(rng, 1, 256)
    budget = (1 << 20) // (c["d"] * c["hkv"] * seqs // 1024 + 1)    # tokens a sequence: at most the listed cases' cache
    c["seqs"] = seqs
    c["hi"] = _log(rng, 16, max(17, min(32768, budget)))
    c["lo"] = max(1, int(c["hi"] * rng.choice([0.05, 0.5, 1.0])))
    if op in ("attend", "weigh", "append"):
        most = max(1, min(c["lo"], 4096 // seqs)) if op != "append" else max(1, min(c["lo"], 32768 // seqs))
        c["qhi"] = 1 if rng.random() < 0.4 else _log(rng, 1, most)
        c["qlo"] = max(1, c["qhi"] // rng.choice([1, 2]))
    if op in ("attend", "weigh"):
        c["hq"] = c["hkv"] * rng.choice([1, 2, 3, 4, 5, 8])
        while c["hq"] * seqs * c["qhi"] * c["hi"] > 32 * 4096 * 8192 and c["qhi"] > 1:
            c["qhi"] = max(1, c["qhi"] // 2)
            c["qlo"] = min(c["qlo"], c["qhi"])
        c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)])
        c["sinks"] = rng.choice([0, 1, 4, 37])
    if op == "evict":
        c["budget"] = _log(rng, 8, max(9, c["hi"]))
        c["sinks"] = rng.randrange(0, c["budget"] // 4 + 1)
        c["recent"] = rng.randrange(0, c["budget"] // 2 + 1)
    return c


def _sizes(c):
    """Lengths of the sequences and numbers of their queries, from the case alone."""
    g = np.random.default_rng(c["seed"])
    lens = g.integers(c["lo"], c["hi"], size=c["seqs"], endpoint=True)
    nq = g.integers(c.get("qlo", 1), c.get("qhi", 1), size=c["seqs"], endpoint=True)
    return lens, np.minimum(nq, lens)


def work(c):
    lens, nq = (x.astype(np.float64) for x in _sizes(c))
    row = c["hkv"] * (c["d"] / 2 + c["d"] / 32)     # a token's K or V in the cache
    n = float(nq.sum())
    if c["op"] == "append":
        return {"bytes": n * (2 * c["hkv"] * c["d"] * 2 + 2 * row + 4 * c["hkv"]), "flops": 0}
    if c["op"] == "evict":
        kept = np.minimum(lens, c["budget"]).sum()
        return {"bytes": float(lens.sum() * c["hkv"] * 4 + kept * (4 * row + c["hkv"] * 8)), "flops": 0}
    seen, pairs = 0.0, 0.0      # tokens that some query sees, and pairs of a query and a token it sees
    for length, m in zip(lens, nq):
        at = length - m + np.arange(m)
        w = c["window"] or length
        lo = np.maximum(at - w + 1, 0)
        s = np.minimum(lo, c["sinks"])
        pairs += float((at - lo + 1 + s).sum())
        seen += length - lo[0] + s[-1] if lo[0] > s[-1] else length
    q = n * c["hq"] * c["d"] * 2
    if c["op"] == "attend":
        return {"bytes": float(seen * 2 * row + 2 * q + n * c["hq"] * 4), "flops": 4 * pairs * c["hq"] * c["d"]}
    return {"bytes": float(seen * (row + 8 * c["hkv"]) + q + n * c["hq"] * 4), "flops": 2 * pairs * c["hq"] * c["d"]}


# ---- the format -----------------------------------------------------------------------------------------------------

def _quantize(x):
    """Codes (two a byte) and scale bytes of [..., D]: blocks of 32, the smallest power of two under which the block's
    largest value still rounds to at most 6, to nearest with ties to the even code."""
    b = x.float().unflatten(-1, (-1, 32))
    bits = b.abs().amax(-1).view(torch.int32)
    byte = ((bits >> 23) - 2 + ((bits & 0x7FFFFF) >= 0x600000).int()).clamp(2, 252)
    a = b.abs() / torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte - 127).unsqueeze(-1)
    code = (a > 0.25).to(torch.uint8)
    for at, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= at) if up else (a > at)
    code |= torch.signbit(b).to(torch.uint8) << 3
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] | (code[..., 1] << 4), byte.to(torch.uint8)


def _values(codes, scales):
    """fp32 [..., D] of bytes [..., D / 2] and scale bytes [..., D / 32]."""
    pair = torch.tensor([[NIBBLE[b & 15], NIBBLE[b >> 4]] for b in range(256)], device=codes.device)
    v = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    return (v * torch.exp2(scales.float() - 127).unsqueeze(-1)).flatten(-2)


def _write(s, page, at, kc, ks, vc, vs):
    """Rows [n, heads, ...] to the slots (page, at)."""
    s["k_codes"][page, :, at] = kc
    s["k_scales"][page, :, at] = ks
    s["v_codes"][page, :, at // 4, :, at % 4] = vc.unflatten(-1, (16, -1))
    s["v_scales"][page, :, :, at] = vs


def _read(s, page, at):
    """What lies at the slots (page, at): K codes and scales, V codes and scales, [..., heads, bytes]."""
    return (s["k_codes"][page, :, at], s["k_scales"][page, :, at],
            s["v_codes"][page, :, at // 4, :, at % 4].flatten(-2), s["v_scales"][page, :, :, at])


# ---- inputs ---------------------------------------------------------------------------------------------------------

def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    lens, nq = _sizes(c)
    h, d, ps = c["hkv"], c["d"], c["page"]
    need = -(-lens // ps)
    width = int(need.max())
    fresh = -(-np.minimum(lens, c["budget"]) // ps) if c["op"] == "evict" else np.zeros_like(need)
    pages = int(need.sum() + fresh.sum()) + 3
    order = torch.randperm(pages, generator=g, device=dev).int()

    def table(counts, first, wide):
        t = torch.zeros(c["seqs"], wide, dtype=torch.int32)
        rows = np.repeat(np.arange(c["seqs"]), counts)
        cols = np.concatenate([np.arange(n) for n in counts]) if counts.sum() else np.zeros(0, np.int64)
        t = t.to(dev)
        t[torch.from_numpy(rows).to(dev), torch.from_numpy(cols).to(dev)] = order[first:first + int(counts.sum())]
        return t

    s = {"case": c, "lens": torch.from_numpy(lens.astype(np.int32)).to(dev), "table": table(need, 0, width),
         "max_len": int(lens.max()), "max_q": int(nq.max()), "total": int(nq.sum()),
         "k_codes": torch.zeros(pages, h, ps, d // 2, dtype=torch.uint8, device=dev),
         "k_scales": torch.zeros(pages, h, ps, d // 32, dtype=torch.uint8, device=dev),
         "v_codes": torch.zeros(pages, h, ps // 4, 16, 4, d // 32, dtype=torch.uint8, device=dev),
         "v_scales": torch.zeros(pages, h, d // 32, ps, dtype=torch.uint8, device=dev),
         "weights": torch.zeros(pages, h, ps, device=dev)}
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    s["cu"] = None if c.get("qhi", 1) == 1 else torch.from_numpy(cu).to(dev)
    # K's channels differ in size, as the key channels of trained models do; V's do not
    sk = torch.exp(0.75 * torch.randn(h, d, generator=g, device=dev))

    if c["op"] == "append":
        n, dt = s["total"], DTYPES[c["dtype"]]
        qkv = torch.randn(n, 4 * h, d, generator=g, device=dev)     # K and V are slices of one projection's output
        qkv[:, 2 * h:3 * h] *= sk
        s["qkv"] = qkv.to(dt)
        s["k"], s["v"] = s["qkv"][:, 2 * h:3 * h], s["qkv"][:, 3 * h:]
    else:
        filled = s["table"].new_zeros(pages, dtype=torch.bool)
        filled[order[:int(need.sum())].long()] = True
        ids = filled.nonzero()[:, 0]
        for part in ids.split(max(1, (1 << 25) // (h * ps * d))):
            shape = (len(part), h, ps, d)
            kc, ks = _quantize((torch.randn(shape, generator=g, device=dev) * sk[:, None]).bfloat16())
            vc, vs = _quantize(torch.randn(shape, generator=g, device=dev).bfloat16())
            s["k_codes"][part], s["k_scales"][part] = kc, ks
            s["v_codes"][part] = vc.unflatten(2, (-1, 4)).unflatten(-1, (16, -1)).transpose(3, 4)
            s["v_scales"][part] = vs.transpose(2, 3)
        # accumulated weights: mostly small, a few large, some equal; what a few queries have left where more are added
        w = (torch.rand(pages, h, ps, generator=g, device=dev) ** 8 * 1024).round() / 64
        s["weights"].copy_(w / c["hi"] if c["op"] == "weigh" else w)
    if c["op"] in ("attend", "weigh"):
        s["scale"] = d ** -0.5
        s["q"] = (torch.randn(s["total"], c["hq"], d, generator=g, device=dev) / (1 + sk.square()).sqrt()
                  .repeat_interleave(c["hq"] // h, 0) * 2).to(DTYPES[c["dtype"]])
    if c["op"] == "weigh":
        s["lse"] = _attend(s, lse_only=True)
    if c["op"] == "evict":
        s["out_table"] = table(fresh, int(need.sum()), int(fresh.max()))
    if own:
        from lossless_bf16_kv_amd import kv4
        s["cache"] = kv4.KV4Cache.from_tensors(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["weights"])
    return s


# ---- the operators --------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        cache = s["cache"]
        mask = {"window": c.get("window") or None, "sinks": c.get("sinks", 0)}
        if c["op"] == "append":
            cache.append(s["k"], s["v"], s["table"], s["lens"], s["cu"])
            return cache.read(s["table"], s["lens"], s["cu"], total=s["total"], dtype=torch.bfloat16)
        if c["op"] == "attend":
            return cache.attend(s["q"], s["table"], s["lens"], s["cu"], max_q=s["max_q"], max_len=s["max_len"],
                                scale=s["scale"], **mask)
        if c["op"] == "weigh":
            cache.weigh(s["q"], s["lse"], s["table"], s["lens"], s["cu"], max_q=s["max_q"], max_len=s["max_len"],
                        scale=s["scale"], **mask)
            return s["weights"]
        out_lens, kept = cache.evict(s["table"], s["lens"], s["out_table"], c["budget"], sinks=c["sinks"],
                                     recent=c["recent"], max_len=s["max_len"])
        return out_lens, kept, s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["weights"]
    if c["op"] == "append":
        return _append(s)
    if c["op"] == "attend":
        return _attend(s)
    if c["op"] == "weigh":
        return _weigh(s)
    return _evict(s)


def _queries(s):
    """Sequence and token position of each query or new token."""
    if s["cu"] is None:
        seq = torch.arange(s["total"], device=s["lens"].device)
        return seq, s["lens"].long() - 1
    cu = s["cu"].long()
    i = torch.arange(s["total"], device=cu.device)
    seq = torch.searchsorted(cu, i, right=True) - 1
    return seq, s["lens"][seq] - (cu[seq + 1] - i)


def _append(s):
    seq, pos = _queries(s)
    ps = s["case"]["page"]
    page, at = s["table"][seq, pos // ps].long(), pos % ps
    _write(s, page, at, *_quantize(s["k"]), *_quantize(s["v"]))
    s["weights"][page, :, at] = 0
    kc, ks, vc, vs = _read(s, page, at)
    return _values(kc, ks).bfloat16(), _values(vc, vs).bfloat16()


def _slots(s):
    """Pages and places in them of the tokens 0 .. longest - 1 of every sequence, and which tokens there are."""
    ps = s["case"]["page"]
    j = torch.arange(s["max_len"], device=s["lens"].device)
    return s["table"][:, j // ps].long(), (j % ps).expand(len(s["lens"]), -1), j, j < s["lens"][:, None]


def _scores(s):
    """Masked scores [seqs, kv_heads, most queries, group, tokens] in fp32, and where in them each query is."""
    c = s["case"]
    page, at, j, there = _slots(s)
    k = _values(s["k_codes"][page, :, at], s["k_scales"][page, :, at]).transpose(1, 2)
    seq, pos = _queries(s)
    row = pos - (s["lens"][seq].long() - s["max_q"])        # the last query of each sequence in the last row
    group = c["hq"] // c["hkv"]
    q = torch.zeros(c["seqs"], s["max_q"], c["hq"], c["d"], device=k.device)
    q[seq, row] = s["q"].float()
    q = q.unflatten(2, (c["hkv"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    a = (q @ k.transpose(2, 3)).mul_(s["scale"]).unflatten(2, (s["max_q"], group))
    i = s["lens"].long()[:, None] - s["max_q"] + torch.arange(s["max_q"], device=k.device)     # positions of the rows
    sees = (j <= i[..., None]) & there[:, None]
    if c["window"]:
        sees &= (j > i[..., None] - c["window"]) | (j < c["sinks"])
    return a.masked_fill_(~sees[:, None, :, None], -math.inf), seq, row


def _attend(s, lse_only=False):
    a, seq, row = _scores(s)
    top = a.amax(-1, keepdim=True).clamp_min_(-1e30)
    p = a.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top)[..., 0].permute(0, 2, 1, 3).flatten(2)[seq, row].contiguous()
    if lse_only:
        return lse
    page, at, _, _ = _slots(s)
    v = _values(s["v_codes"][page, :, at // 4, :, at % 4].flatten(-2), s["v_scales"][page, :, :, at]).transpose(1, 2)
    o = (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4]) / total.clamp_min(1e-30)
    return o.permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, row].to(s["q"].dtype), lse


def _weigh(s):
    c = s["case"]
    a, seq, row = _scores(s)
    lse = a.new_full((c["seqs"], s["max_q"], c["hq"]), math.inf)
    lse[seq, row] = s["lse"]
    lse = lse.unflatten(2, (c["hkv"], -1)).permute(0, 2, 1, 3)[..., None]
    w = a.sub_(lse).exp_().sum((2, 3)).transpose(1, 2)      # [seqs, tokens, kv_heads]
    page, at, _, there = _slots(s)
    s["weights"][page[there], :, at[there]] += w[there]
    return s["weights"]


def _evict(s):
    c = s["case"]
    page, at, j, there = _slots(s)
    n, budget, ps = s["lens"].long()[:, None], c["budget"], c["page"]
    w = s["weights"][page, :, at].transpose(1, 2)           # [seqs, kv_heads, tokens]
    rank = torch.where(there & (j < c["sinks"]) | (j >= n - c["recent"]), math.inf, 0)[:, None] + w
    rank = rank.masked_fill(~there[:, None], -math.inf)
    take = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    out_lens = s["lens"].clamp_max(budget)
    late = torch.arange(take.shape[-1], device=n.device) >= out_lens[:, None, None]
    kept = take.masked_fill(late, 1 << 30).sort(-1).values
    full = torch.full((*kept.shape[:2], budget), -1, dtype=torch.int32, device=n.device)
    full[..., :kept.shape[-1]] = kept.masked_fill(late, -1).int()
    # every kept (sequence, head, token) moves to its new slot
    seq, head, to = (~late).expand(kept.shape).nonzero(as_tuple=True)
    old = kept[seq, head, to]
    a, b = s["table"][seq, old // ps].long(), old % ps
    x, y = s["out_table"][seq, to // ps].long(), to % ps
    for name in ("k_codes", "k_scales", "weights"):
        s[name][x, head, y] = s[name][a, head, b]
    s["v_codes"][x, head, y // 4, :, y % 4] = s["v_codes"][a, head, b // 4, :, b % 4]
    s["v_scales"][x, head, :, y] = s["v_scales"][a, head, :, b]
    return out_lens, full, s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["weights"]


# ---- the definition in 64 bits --------------------------------------------------------------------------------------

def _round64(x):
    """What a [n, heads, D] tensor reads as after its way through the format, by the nearest value of the grid."""
    b = x.double().unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))      # largest value = m 2^e, m in [0.5, 1)
    e = (e - 3 + (m >= 0.875).int()).clamp(2 - 127, 252 - 127)
    a = torch.ldexp(b, -e)
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
    return torch.ldexp((a / step).round() * step, e).clamp(-6.0 * 2.0 ** 125, 6.0 * 2.0 ** 125).flatten(-2)


def _head64(s, q, head, tokens):
    """K and V of one sequence's head in 64 bits, byte by byte."""
    c = s["case"]
    t = torch.arange(tokens, device=s["lens"].device)
    page, at = s["table"][q, t // c["page"]].long(), t % c["page"]
    grid = torch.tensor(NIBBLE, dtype=torch.float64, device=t.device)
    vc = s["v_codes"][page, head][t, at // 4, :, at % 4].flatten(1)
    out = []
    for codes, scales in ((s["k_codes"][page, head, at], s["k_scales"][page, head, at]),
                          (vc, s["v_scales"][page, head, :, at])):
        v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).flatten(1)
        out.append(v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1))
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "append":
        return _round64(s["k"]), _round64(s["v"])
    lens, nq = _sizes(c)
    if c["op"] == "evict" or c["seqs"] * c["hkv"] > 3000:
        return None
    group, cu = c["hq"] // c["hkv"], np.concatenate([[0], np.cumsum(nq)])
    out = torch.zeros(s["total"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], c["hq"], dtype=torch.float64, device="cuda")
    weights = s["weights"].double()
    for b in range(c["seqs"]):
        n, m, r = int(lens[b]), int(nq[b]), slice(int(cu[b]), int(cu[b + 1]))
        j = torch.arange(n, device="cuda")
        i = n - m + torch.arange(m, device="cuda")[:, None]
        hidden = j > i
        if c["window"]:
            hidden = hidden | ((i - j >= c["window"]) & (j >= c["sinks"]))
        page, at = s["table"][b, j // c["page"]].long(), j % c["page"]
        for h in range(c["hkv"]):
            k, v = _head64(s, b, h, n)
            for f in range(h * group, (h + 1) * group):
                a = (s["q"][r, f].double() @ k.T) * s["scale"]
                a[hidden] = -math.inf
                if c["op"] == "attend":
                    lse[r, f] = torch.logsumexp(a, 1)
                    out[r, f] = torch.softmax(a, 1) @ v
                else:
                    weights[page, h, at] += torch.exp(a - s["lse"][r, f, None].double()).sum(0)
    return (out, lse) if c["op"] == "attend" else weights
