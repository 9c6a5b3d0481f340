"""The operators between the quantized projections of a serving step, as cases to be measured.

A decode step of this library's projections (q/k/v, o, gate/up/down, lm_head) needs four things around them:
rotary positions on q and k, the new keys and values put into an 8-bit paged cache, attention over that cache,
and the draw of the next token from the logits.  Each case is one call of one of them:

    rope     q and k rotated by position, interleaved or half layout, the whole head or its first part
    append   new k and v quantized into the cache: int8 codes, one scale for each block of tokens and head
    attend   causal attention of new tokens (one for each sequence, or a prompt's chunk) over that cache
    sample   temperature, top-k, top-p and min-p, then a draw from given uniform numbers

``run`` computes a case in plain torch operations where ``own`` is false, and by the library's entry points where
it is true.  The cache's layout: k codes int8 [blocks, kv heads, block, head dim], v codes int8 [blocks, kv heads,
head dim, block], scales f32 [blocks, kv heads]; a sequence's block j is ``table[s, j]``; a code c stands for c * scale.
"""

import math
import random

import torch

own = False

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's chat on a small model: one new token, a short odd context, small pages (latency)
        dict(name="attend-one", op="attend", seqs=1, new="one", lo=777, hi=777, heads=32, kv_heads=8, dim=64, block=16,
             window=0, lse=False, type="f16"),
        # a serving batch: one new token for each of 64 sequences, contexts from a few tokens to 8192
        dict(name="attend-batch", op="attend", seqs=64, new="one", lo=5, hi=8192, heads=32, kv_heads=8, dim=128, block=64,
             window=0, lse=False, type="bf16"),
        # two long documents: the axis that has to be split
        dict(name="attend-long", op="attend", seqs=2, new="one", lo=131000, hi=131071, heads=32, kv_heads=8, dim=128,
             block=32, window=0, lse=False, type="f16"),
        # a fresh prompt of odd length on a small model
        dict(name="attend-prompt", op="attend", seqs=1, new="all", lo=4001, hi=4001, heads=32, kv_heads=8, dim=64, block=64,
             window=0, lse=False, type="f16"),
        # chunks of up to 1024 prompt tokens over cached prefixes, a sliding window, the log-sum kept for a later merge
        dict(name="attend-chunks", op="attend", seqs=6, new="1024", lo=900, hi=8192, heads=32, kv_heads=8, dim=128, block=64,
             window=4096, lse=True, type="bf16"),
        # one new token of each of 8 sequences at far positions, frequencies scaled for a long context
        dict(name="rope-decode", op="rope", tokens=8, far=131072, heads=32, kv_heads=8, dim=64, rot=64, interleaved=False,
             scaled=True, type="f16"),
        # a prompt's q and k out of the fused projection, half of each head rotated, pairs interleaved
        dict(name="rope-prompt", op="rope", tokens=8191, far=8192, heads=32, kv_heads=8, dim=128, rot=64, interleaved=True,
             scaled=False, type="bf16"),
        # one new token for each of 256 sequences, most of them into a block that is partly filled
        dict(name="append-decode", op="append", seqs=256, new="one", lo=1, hi=700, kv_heads=8, dim=128, block=64, type="bf16"),
        # prompts' chunks, starting and ending inside a block
        dict(name="append-prompt", op="append", seqs=5, new="4096", lo=300, hi=8192, kv_heads=8, dim=64, block=32, type="f16"),
        # one user's next token from the 128256 logits of lm_head (latency)
        dict(name="sample-one", op="sample", rows=1, vocab=128256, temperature=0.8, top_k=40, top_p=0.95, min_p=0.0,
             mixed=False, type="f16"),
        # a serving batch, every row with settings of its own (greedy, filters off and on)
        dict(name="sample-batch", op="sample", rows=192, vocab=128256, temperature=1.0, top_k=0, top_p=0.9, min_p=0.0,
             mixed=True, type="f16"),
        # a smaller vocabulary of odd size, 32-bit logits, min-p alone
        dict(name="sample-odd", op="sample", rows=17, vocab=32003, temperature=1.3, top_k=0, top_p=1.0, min_p=0.02,
             mixed=False, type="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "chunks", "chunks", "rope", "append", "sample", "sample"])
    kv_heads, group = rng.choice([(1, 8), (2, 5), (4, 4), (8, 1), (8, 4), (8, 8)])
    dim, block, t = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice(["f16", "bf16"])
    if kind == "decode":
        hi = _log(rng, 3, 131071)
        seqs = _log(rng, 1, max(1, min(128, 270000 // hi)))
        return dict(op="attend", seqs=seqs, new=rng.choice(["one", "one", "5"]), lo=max(1, int(hi * rng.choice([0.01, 0.5, 1]))),
                    hi=hi, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, block=block,
                    window=rng.choice([0, 0, 0, 1000]), lse=rng.random() < 0.3, type=t)
    if kind == "chunks":
        hi = _log(rng, 17, 8192)
        new = _log(rng, 9, 1024)
        return dict(op="attend", seqs=_log(rng, 1, max(1, min(6, 11000000 // (hi * new)))), new=str(new), lo=max(1, hi // rng.choice([1, 3, 20])), hi=hi,
                    heads=min(32, kv_heads * group), kv_heads=min(8, kv_heads), dim=dim, block=block,
                    window=rng.choice([0, 0, 513]), lse=rng.random() < 0.3, type=t)
    if kind == "rope":
        return dict(op="rope", tokens=_log(rng, 1, 8191), far=_log(rng, 8192, 131072), heads=min(32, kv_heads * group),
                    kv_heads=min(8, kv_heads), dim=dim, rot=rng.choice([dim, dim // 2, dim // 4]),
                    interleaved=rng.random() < 0.5, scaled=rng.random() < 0.5, type=t)
    if kind == "append":
        one = rng.random() < 0.5
        hi = _log(rng, 2, 700 if one else 8192)
        return dict(op="append", seqs=_log(rng, 1, 256 if one else 5), new="one" if one else str(_log(rng, 3, 4096)),
                    lo=max(1, hi // 10), hi=hi, kv_heads=kv_heads, dim=dim, block=block, type=t)
    vocab = _log(rng, 1000, 128256)
    return dict(op="sample", rows=_log(rng, 1, 192), vocab=vocab, temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.7]),
                top_k=rng.choice([0, 0, 1, 20, 500, 20000]), top_p=rng.choice([1.0, 1.0, 0.5, 0.9, 0.99]),
                min_p=rng.choice([0.0, 0.0, 0.05, 0.3]), mixed=rng.random() < 0.3, type=rng.choice(["f16", "bf16", "f32"]))


def _lengths(case):
    """Each sequence's length with its new tokens, and how many are new: plain numbers, the case's own."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k not in ("name", "type"))))
    lens = [_log(rng, case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if case["new"] == "one":
        return lens, [1] * len(lens)
    if case["new"] == "all":
        return lens, list(lens)
    most = int(case["new"])
    return lens, [min(n, most if most <= 8 else rng.randint(max(1, most // 2), most)) for n in lens]


# ------------------------------------------------------------------------------------------------ inputs
def _paged(case, lens, gen):
    """A pool of blocks in shuffled order and the sequences' table; entries past a sequence's end are -1."""
    counts = [-(-n // case["block"]) for n in lens]
    total = sum(counts)
    ids = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    width = max(counts)
    at = torch.tensor([sum(counts[:i]) for i in range(len(counts))], device=DEV)[:, None] + torch.arange(width, device=DEV)
    used = torch.arange(width, device=DEV) < torch.tensor(counts, device=DEV)[:, None]
    return total, torch.where(used, ids[at.clamp(max=total - 1)], -1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = dict(case=case)
    if case["op"] == "rope":
        n, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        qkv = normal(n, (h + 2 * hk) * d).to(t)           # the fused projection's output: q and k are views of it
        s["q"] = qkv[:, :h * d].view(n, h, d)
        s["k"] = qkv[:, h * d:(h + hk) * d].view(n, hk, d)
        first = torch.randint(0, max(1, case["far"] - n), (1,), generator=gen, device=DEV)
        s["positions"] = ((first + torch.arange(n, device=DEV)) if n > 64 else
                          torch.randint(0, case["far"], (n,), generator=gen, device=DEV)).to(torch.int32)
        f = 500000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
        if case["scaled"]:                                # low frequencies slowed eightfold, high ones kept, blended between
            turns = 8192 * f / (2 * math.pi)
            keep = ((turns - 1) / (4 - 1)).clamp(0, 1)
            f = keep * f + (1 - keep) * f / 8
        s["inv_freq"] = f.to(torch.float32).to(DEV)
        return s
    if case["op"] == "sample":
        r, v = case["rows"], case["vocab"]
        x = normal(r, v) * 2.5
        likely = torch.randint(0, v, (r, 12), generator=gen, device=DEV)
        x.scatter_add_(1, likely, 6 + 2 * normal(r, 12))  # a few likely tokens over a broad rest
        s["logits"] = x.to(t)
        s["u"] = torch.rand(r, generator=gen, device=DEV)
        at = torch.arange(r, device=DEV)
        pick = (lambda a, *vals: torch.tensor(vals, device=DEV)[at % len(vals)] if case["mixed"] else torch.full((r,), a, device=DEV))
        s["temperature"] = pick(case["temperature"], 0.7, 1.0, 0.0, 1.5, 0.9).to(torch.float32)
        s["top_k"] = pick(case["top_k"], 0, 50, 0, 1000).to(torch.int32)
        s["top_p"] = pick(case["top_p"], 0.9, 1.0, 0.95).to(torch.float32)
        s["min_p"] = pick(case["min_p"], 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.05).to(torch.float32)
        return s
    lens, new = _lengths(case)
    hk, d, b = case["kv_heads"], case["dim"], case["block"]
    blocks, s["table"] = _paged(case, lens, gen)
    # codes and scales as a normal k and v leave them: the block's largest value near three and a half deviations
    s["k_codes"] = (normal(blocks, hk, b, d) * 36).round_().clamp_(-127, 127).to(torch.int8)
    s["v_codes"] = (normal(blocks, hk, d, b) * 36).round_().clamp_(-127, 127).to(torch.int8)
    s["k_scale"] = 0.02 + 0.015 * torch.rand(blocks, hk, generator=gen, device=DEV)
    s["v_scale"] = 0.02 + 0.015 * torch.rand(blocks, hk, generator=gen, device=DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["starts"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    s["most_new"], s["longest"], n = max(new), max(lens), sum(new)
    if case["op"] == "attend":
        s["q"] = normal(n, case["heads"], d).to(t)
    else:
        kv = normal(n, 2 * hk * d).to(t)
        s["k"], s["v"] = kv[:, :hk * d].view(n, hk, d), kv[:, hk * d:].view(n, hk, d)
    return s


# --------------------------------------------------------------------------------------------------- run
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_cache(s):
    import dequant_matmul_qmv_amd as mxq
    return mxq.KvCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])


def _own_rope(s):
    import dequant_matmul_qmv_amd as mxq
    return mxq.mxq_rope(s["q"], s["k"], s["inv_freq"], s["positions"], interleaved=s["case"]["interleaved"])


def _own_append(s):
    import dequant_matmul_qmv_amd as mxq
    c = mxq.mxq_kv_append(_own_cache(s), s["k"], s["v"], s["table"], s["lens"],
                          None if s["case"]["new"] == "one" else s["starts"])
    return c.k, c.v, c.k_scale, c.v_scale


def _own_attend(s):
    import dequant_matmul_qmv_amd as mxq
    return mxq.mxq_attention(s["q"], _own_cache(s), s["table"], s["lens"],
                             None if s["case"]["new"] == "one" else s["starts"], window=s["case"]["window"],
                             return_lse=s["case"]["lse"])


def _own_sample(s):
    import dequant_matmul_qmv_amd as mxq
    return mxq.mxq_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                          min_p=s["min_p"])


_run_own = {"rope": _own_rope, "append": _own_append, "attend": _own_attend, "sample": _own_sample}


def _plain_rope(s):
    case, rot = s["case"], s["case"]["rot"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()        # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        y = x.float()
        if case["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((z.to(x.dtype), x[..., rot:]), -1)

    return turn(s["q"]), turn(s["k"])


def _token_places(s):
    """For each new token: its sequence, its number among the sequence's new ones, its position."""
    starts, lens = s["starts"].long(), s["lens"].long()
    n = (s["k"] if "k" in s else s["q"]).shape[0]
    t = torch.arange(n, device=DEV)
    seq = torch.searchsorted(starts[1:], t, right=True)
    nth = t - starts[seq]
    return seq, nth, lens[seq] - (starts[seq + 1] - starts[seq]) + nth


def _plain_append(s):
    b = s["case"]["block"]
    seq, _, pos = _token_places(s)
    block, slot = s["table"][seq, pos // b].long(), pos % b
    first = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1])          # tokens that were there before
    part = torch.gather(s["table"], 1, (first // b).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    held = torch.where(part >= 0, first % b, 0)                              # ... of them in the block that is continued
    part = part.clamp(min=0)

    def put(codes, scale, x, by_token):
        x = x.float()
        fresh = torch.zeros_like(scale).index_reduce_(0, block, x.abs().amax(-1), "amax")
        was = torch.zeros_like(scale)
        was[part] = torch.where(held[:, None] > 0, scale[part], 0.0)
        # quotients in 64 bits, rounded once: a 32-bit quotient is then the nearest one whatever the divider
        wide = torch.maximum(was, (fresh.double() / 127).float())
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEV)
        touched[block] = True
        scale.copy_(torch.where(touched[:, None], wide, scale))
        ratio = torch.where(wide > 0, was.double() / wide.double(), 0.0).float()[part][..., None, None]
        old = codes[part]
        keep = (torch.arange(b, device=DEV) < held[:, None])[:, None]
        keep = keep[..., None] if by_token else keep[:, :, None]
        codes[part] = torch.where(keep, (old.float() * ratio).round().to(torch.int8), old)
        inv = torch.where(wide > 0, 1 / wide.double(), 0.0).float().clamp(max=torch.finfo(torch.float32).max)
        c = (x * inv[block][..., None]).round().clamp(-127, 127).to(torch.int8)
        if by_token:
            codes[block, :, slot] = c
        else:
            codes[block, :, :, slot] = c

    put(s["k_codes"], s["k_scale"], s["k"], True)
    put(s["v_codes"], s["v_scale"], s["v"], False)
    return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]


def _plain_attend(s):
    case = s["case"]
    hk, g, d, b = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], case["block"]
    n, most, width = case["seqs"], s["most_new"], -(-s["longest"] // case["block"])
    ids = s["table"][:, :width].long().clamp(min=0)
    k = s["k_codes"][ids].float() * s["k_scale"][ids][..., None, None]       # [seqs, width, hk, b, d]
    v = s["v_codes"][ids].float() * s["v_scale"][ids][..., None, None]       # [seqs, width, hk, d, b]
    k = k.permute(0, 2, 1, 3, 4).reshape(n, hk, width * b, d)
    v = v.permute(0, 2, 1, 4, 3).reshape(n, hk, width * b, d)
    starts, lens = s["starts"].long(), s["lens"].long()
    new = starts[1:] - starts[:-1]
    nth = torch.arange(most, device=DEV)
    rows = (starts[:-1, None] + nth).clamp(max=s["q"].shape[0] - 1)          # the shorter ones repeat rows that are not kept
    q = s["q"][rows].float().view(n, most, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * most, d)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(n, hk, g, most, width * b)
    pos = (lens - new)[:, None] + nth
    at = torch.arange(width * b, device=DEV)
    seen = (at <= pos[..., None]) & (at < lens[:, None, None])
    if case["window"]:
        seen &= at > pos[..., None] - case["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top.isfinite(), top, 0.0)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    y = torch.matmul(p.view(n, hk, g * most, width * b), v).view(n, hk, g, most, d)
    y = torch.where(total > 0, y / total, 0.0)
    seq, nth, _ = _token_places(s)
    out = y.permute(0, 3, 1, 2, 4).reshape(n, most, hk * g, d)[seq, nth].to(s["q"].dtype)
    if not case["lse"]:
        return out
    return out, (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(n, most, hk * g)[seq, nth]


def _plain_sample(s):
    x = s["logits"].double()                              # 64 bits: which token a border falls on is a whole number
    x = torch.where(x.isnan(), -math.inf, x)
    x, order = x.sort(dim=1, descending=True, stable=True)
    top, t = x[:, :1], s["temperature"].double()[:, None]
    w = torch.where(x == top, 1.0, ((x - top) / t).exp())
    w = torch.where((t > 0) | (x == top), w, 0.0)
    rank = torch.arange(x.shape[1], device=DEV)
    k = torch.where(t > 0, s["top_k"].long()[:, None], 1)  # temperature 0: the largest, the first of equals
    w = torch.where((k <= 0) | (rank < k), w, 0.0)
    p = s["top_p"].double()[:, None]
    sums = w.cumsum(1)
    before = torch.cat((torch.zeros_like(top), sums[:, :-1]), 1)
    w = torch.where((p >= 1) | (rank == 0) | (before < p * sums[:, -1:]), w, 0.0)
    w = torch.where((rank == 0) | (w >= s["min_p"].double()[:, None]), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)         # back in the tokens' order
    sums = w.cumsum(1)
    total = sums[:, -1:]
    token = torch.searchsorted(sums, s["u"].double()[:, None] * total, right=True).clamp(max=x.shape[1] - 1)
    prob = w.gather(1, token) / total
    return token[:, 0].to(torch.int32), prob[:, 0].float()


_run_plain = {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}


# -------------------------------------------------------------------------------------------------- work
def work(case):
    e = TYPES[case["type"]].itemsize
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * n * case["dim"] * e + 4 * case["tokens"] + 2 * case["rot"], "flops": 3 * n * case["rot"]}
    if case["op"] == "sample":                            # one exponential and one comparison for each logit at the least
        n = case["rows"] * case["vocab"]
        return {"bytes": n * e + case["rows"] * 28, "flops": 2 * n}
    lens, new = _lengths(case)
    hk, d = case["kv_heads"], case["dim"]
    if case["op"] == "append":                            # the new tokens read and their codes written
        n = sum(new) * hk * d * 2
        return {"bytes": n * (e + 1), "flops": 3 * n}
    tokens = pairs = 0
    for length, n in zip(lens, new):
        w = case["window"] or length
        tokens += min(length, w + n - 1)
        full = max(0, min(n, length - w))                 # rows whose window is full
        rest = n - full                                   # the others see 1 + length - n .. tokens
        pairs += full * w + rest * (length - n) + rest * (rest + 1) // 2
    bytes_ = 2 * tokens * hk * (d + 4 / case["block"]) + 2 * sum(new) * case["heads"] * d * e
    return {"bytes": bytes_, "flops": 4 * pairs * case["heads"] * d}


# ------------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions, token by token or sequence by sequence, in 64 bits."""
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](case, s)


def _exact_rope(case, s):
    """(a + ib) times e^(i angle), for each pair."""
    rot, half = case["rot"], case["rot"] // 2
    i = torch.arange(half, device=DEV)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, half + i)
    angle = torch.outer(s["positions"].to(torch.float64), s["inv_freq"].to(torch.float64))
    unit = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    out = []
    for x in (s["q"], s["k"]):
        y = x.to(torch.float64).clone()
        z = torch.complex(y[..., first], y[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_append(case, s):
    """The scales in 64 bits; codes are whole numbers that the 32-bit rule alone defines, so they have no such value."""
    b, lens, new = case["block"], *_lengths(case)
    table = s["table"].cpu()
    scales = []
    for name, x in (("k_scale", s["k"]), ("v_scale", s["v"])):
        peak = x.to(torch.float64).abs().amax(-1).cpu()
        scale = s[name].to(torch.float64).cpu()
        at = 0
        for i, (length, n) in enumerate(zip(lens, new)):
            begin = length - n
            for j in range(begin // b, -(-length // b)):
                lo, hi = max(begin, j * b), min(length, (j + 1) * b)
                got = peak[at + lo - begin:at + hi - begin].amax(0) / 127
                row = scale[table[i, j]]
                scale[table[i, j]] = torch.maximum(row, got) if j * b < begin else got
            at += n
        scales.append(scale)
    return None, None, scales[0], scales[1]


def _exact_attend(case, s):
    b, hk, d = case["block"], case["kv_heads"], case["dim"]
    g = case["heads"] // hk
    lens, new = _lengths(case)
    out, lse, at = [], [], 0
    for i, (length, n) in enumerate(zip(lens, new)):
        ids = s["table"][i, :-(-length // b)].long()
        q = s["q"][at:at + n].double() / math.sqrt(d)
        pos = torch.arange(length - n, length, device=DEV)[:, None]
        key = torch.arange(length, device=DEV)[None, :]
        hide = (key > pos) | ((key <= pos - case["window"]) if case["window"] else False)
        ys, ls = [], []
        for h in range(hk):
            k = (s["k_codes"][ids, h].double() * s["k_scale"][ids, h].double()[:, None, None]).flatten(0, 1)[:length]
            v = (s["v_codes"][ids, h].double() * s["v_scale"][ids, h].double()[:, None, None]).transpose(1, 2).flatten(0, 1)[:length]
            for j in range(g):
                x = (q[:, h * g + j] @ k.T).masked_fill(hide, -math.inf)
                ls.append(x.logsumexp(-1))
                ys.append((x - ls[-1][:, None]).exp() @ v)
        out.append(torch.stack(ys, 1))
        lse.append(torch.stack(ls, 1))
        at += n
    return (torch.cat(out), torch.cat(lse)) if case["lse"] else torch.cat(out)


def _exact_sample(case, s):
    """Row by row: the tokens in descending order, cut to the shortest of the three prefixes, one drawn in token order."""
    tokens, probs = [], []
    for r in range(case["rows"]):
        x = s["logits"][r].double()
        t = s["temperature"][r].item()
        if t <= 0:
            tokens.append(int((x == x.max()).nonzero()[0]))
            probs.append(1.0)
            continue
        z = torch.softmax(x / t, 0)
        z, order = z.sort(descending=True, stable=True)
        keep = z.numel() if s["top_k"][r] <= 0 else min(z.numel(), int(s["top_k"][r]))
        if s["top_p"][r] < 1:
            mass = z[:keep].cumsum(0)
            keep = min(keep, 1 + int((mass < s["top_p"][r].double() * mass[-1]).sum()))
        keep = max(1, min(keep, int((z >= s["min_p"][r].double() * z[0]).sum())))
        kept = order[:keep].sort()
        z = z[:keep][kept.indices]
        mass = z.cumsum(0)
        at = min(keep - 1, int((mass <= s["u"][r].double() * mass[-1]).sum()))
        tokens.append(int(kept.values[at]))
        probs.append(float(z[at] / mass[-1]))
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64)
