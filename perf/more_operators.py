"""The way from the fused q/k/v projection to attention's output over a cache held in 4 bits, as cases to be measured.

Three operators, each case one call of one of them:

    turn     q and k normed head by head (root mean square, a weight for each value) and rotated by position in the
             same pass; a pair turns by one of several axes' positions (time, height, width)
    append   new keys normed, rotated and quantized into a paged cache of 8 or 4 bits together with the new values,
             and q normed and rotated beside them
    attend   causal attention of new tokens (one for each sequence, or a prompt's chunk) over the cache of 4 bits

``run`` computes a case in plain torch operations where ``own`` is false, and by the library's entry points where it
is true.  A sequence's tokens ``j * block ..`` are in the page ``table[s, j]``.  The cache of 8 bits: k codes int8
[blocks, kv heads, block, dim], v codes int8 [blocks, kv heads, dim, block], scales f32 [blocks, kv heads].  The cache
of 4 bits: a value is (code - zero) * scale, with a scale and a zero point for each token and kv head; k words int32
[blocks, kv heads, block, dim / 8] hold 8 values of a token, v words int32 [blocks, kv heads, block / 8, dim] hold one
value of 8 tokens, lowest bits first; the scale's int16 word is an f16 number of 7 significant bits whose lowest 4
bits are the zero point.  Codes and scales are returned as they are held: whole numbers, by a rule that leaves none of
their roundings open.
"""

import math
import random

import torch

own = False

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of each of 8 sequences at far positions, both norms (latency)
        dict(name="turn-decode", op="turn", tokens=8, far=131072, axes=1, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, type="bf16"),
        # a prompt's q and k as views of the fused projection, both norms
        dict(name="turn-prompt", op="turn", tokens=8191, far=8192, axes=1, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, type="bf16"),
        # frames of a video: positions of time, height and width, half of each head rotated, pairs interleaved
        dict(name="turn-video", op="turn", tokens=5003, far=600, axes=3, heads=16, kv_heads=4, dim=64, rot=32,
             interleaved=True, norm=True, type="f16"),
        # a serving batch's decode step into the cache of 8 bits
        dict(name="append8-decode", op="append", bits=8, seqs=256, new="one", lo=1, hi=700, heads=32, kv_heads=8, dim=128,
             rot=128, block=64, axes=1, implied=True, interleaved=False, norm=True, type="bf16"),
        # prompts' chunks into the cache of 8 bits, starting and ending inside a page, no norms
        dict(name="append8-prompt", op="append", bits=8, seqs=5, new="4096", lo=300, hi=8192, heads=32, kv_heads=4, dim=64,
             rot=64, block=32, axes=1, implied=False, interleaved=False, norm=False, type="f16"),
        # a decode step into the cache of 4 bits: far positions given by the caller
        dict(name="append4-decode", op="append", bits=4, seqs=64, new="one", lo=5, hi=8192, heads=32, kv_heads=8, dim=128,
             rot=128, block=64, axes=1, implied=False, interleaved=False, norm=True, type="f16"),
        # prompts' chunks into the cache of 4 bits, both norms
        dict(name="append4-prompt", op="append", bits=4, seqs=5, new="4096", lo=300, hi=8192, heads=32, kv_heads=8, dim=128,
             rot=128, block=64, axes=1, implied=True, interleaved=False, norm=True, type="bf16"),
        # one user's chat on a small model: a short odd context, small pages (latency)
        dict(name="attend4-one", op="attend", seqs=1, new="one", lo=913, hi=913, heads=32, kv_heads=8, dim=64, block=16,
             window=0, lse=False, type="f16"),
        # a serving batch: one new token for each of 96 sequences, contexts from a few tokens to 8192
        dict(name="attend4-batch", op="attend", seqs=96, new="one", lo=5, hi=8192, heads=32, kv_heads=8, dim=128, block=64,
             window=0, lse=False, type="bf16"),
        # three long documents, which is what a cache of 4 bits is for
        dict(name="attend4-long", op="attend", seqs=3, new="one", lo=131000, hi=131071, heads=32, kv_heads=8, dim=128,
             block=32, window=0, lse=False, type="f16"),
        # a fresh prompt of odd length on a small model
        dict(name="attend4-prompt", op="attend", seqs=1, new="all", lo=4001, hi=4001, heads=32, kv_heads=8, dim=64, block=64,
             window=0, lse=False, type="f16"),
        # chunks of up to 1024 prompt tokens over cached prefixes, a sliding window, the log-sum kept for a later merge
        dict(name="attend4-chunks", op="attend", seqs=6, new="1024", lo=900, hi=8192, heads=32, kv_heads=8, dim=128, block=64,
             window=4096, lse=True, type="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "chunks", "chunks", "turn", "append one", "append many"])
    kv_heads, group = rng.choice([(1, 8), (2, 5), (4, 4), (8, 1), (8, 4), (8, 8)])
    dim, block, t = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice(["f16", "bf16"])
    if kind == "decode":
        hi = _log(rng, 3, 131071)
        seqs = _log(rng, 1, max(1, min(128, 390000 // hi)))
        return dict(op="attend", seqs=seqs, new=rng.choice(["one", "one", "5"]), lo=max(1, int(hi * rng.choice([0.01, 0.5, 1]))),
                    hi=hi, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, block=block,
                    window=rng.choice([0, 0, 0, 1000]), lse=rng.random() < 0.3, type=t)
    if kind == "chunks":
        hi = _log(rng, 17, 8192)
        new = _log(rng, 9, 1024)
        return dict(op="attend", seqs=_log(rng, 1, max(1, min(6, 11000000 // (hi * new)))), new=str(new),
                    lo=max(1, hi // rng.choice([1, 3, 20])), hi=hi, heads=min(32, kv_heads * group), kv_heads=min(8, kv_heads),
                    dim=dim, block=block, window=rng.choice([0, 0, 513]), lse=rng.random() < 0.3, type=t)
    heads, norm = min(32, kv_heads * group), rng.random() < 0.6
    dim = rng.choice([64, 128, 256]) if kind == "turn" else dim
    rot, inter = rng.choice([dim, dim, dim // 2, dim // 4]), rng.random() < 0.4
    if kind == "turn":
        axes = rng.choice([1, 1, 2, 3])
        return dict(op="turn", tokens=_log(rng, 1, 8191), far=_log(rng, 600, 131072), axes=axes, heads=heads, kv_heads=kv_heads,
                    dim=dim, rot=rot, interleaved=inter, norm=norm, type=t)
    one, axes = kind == "append one", rng.choice([1, 1, 1, 3])
    hi = _log(rng, 2, 8192)
    return dict(op="append", bits=rng.choice([4, 4, 8]), seqs=_log(rng, 1, min(256, max(1, 400000 // hi)) if one else 5),
                new="one" if one else str(_log(rng, 3, 4096)), lo=max(1, hi // 10), hi=hi, heads=heads, kv_heads=kv_heads,
                dim=dim, rot=rot, block=block, axes=axes, implied=axes == 1 and rng.random() < 0.5, interleaved=inter,
                norm=norm, type=t)


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


def _words(gen, *shape):
    """Words of 8 codes, each the sum of two uniform numbers of 3 bits and one of 1: a hill around 7.5, as values leave it."""
    def bits(mask):
        return torch.randint(-2 ** 31, 2 ** 31, shape, generator=gen, device=DEV, dtype=torch.int64).to(torch.int32) & mask
    return bits(0x77777777) + bits(0x77777777) + bits(0x11111111)


def _scales(gen, *shape):
    """Scale words: 7 bits of a scale near a fifteenth of a normal value's range, and a zero point near the middle."""
    s = (0.22 + 0.16 * torch.rand(*shape, generator=gen, device=DEV)).to(torch.float16).view(torch.int16) & 0x7FF0
    return s | torch.randint(5, 11, shape, generator=gen, device=DEV, dtype=torch.int16)


def _turning(case, n, gen, s):
    """Frequencies, weights and (unless a token's place is its position) positions."""
    rot, half = case["rot"], case["rot"] // 2
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    s["inv_freq"] = f.to(torch.float32).to(DEV)
    s["axes"], s["q_weight"], s["k_weight"] = None, None, None
    if case["axes"] > 1:                                  # the first pairs turn by time, the others by height and width
        cut = [half // 4, half // 4 + (half - half // 4) // 2] if case["axes"] == 3 else [half // 2]
        s["axes"] = torch.bucketize(torch.arange(half), torch.tensor(cut), right=True).to(torch.int32).to(DEV)
    if case["norm"]:
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.randn(case["dim"], generator=gen, device=DEV)).to(TYPES[case["type"]])
                                        for _ in range(2))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = dict(case=case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "turn":
        n = case["tokens"]
        qkv = (normal(n, (h + 2 * hk) * d) * 1.5).to(t)   # the fused projection's output: q and k are views of it
        s["q"] = qkv[:, :h * d].view(n, h, d)
        s["k"] = qkv[:, h * d:(h + hk) * d].view(n, hk, d)
        _turning(case, n, gen, s)
        far = case["far"]
        if case["axes"] > 1:                              # a video's patches: rows of 40 by 30, frame after frame
            at = torch.arange(n, device=DEV) + torch.randint(0, far, (1,), generator=gen, device=DEV)
            grid = torch.stack((at // 1200, at % 1200 // 40, at % 40))
            s["positions"] = (grid if case["axes"] == 3 else grid[1:]).to(torch.int32).contiguous()
        else:
            first = torch.randint(0, max(1, far - n), (1,), generator=gen, device=DEV)
            s["positions"] = ((first + torch.arange(n, device=DEV)) if n > 64 else
                              torch.randint(0, far, (n,), generator=gen, device=DEV)).to(torch.int32)
        return s
    lens, new = _lengths(case)
    b, n = case["block"], sum(new)
    blocks, s["table"] = _paged(case, lens, gen)
    if case["op"] == "append" and case["bits"] == 8:
        s["k_codes"] = (normal(blocks, hk, b, d) * 36).round_().clamp_(-127, 127).to(torch.int8)
        s["v_codes"] = (normal(blocks, hk, d, b) * 36).round_().clamp_(-127, 127).to(torch.int8)
        s["k_scale"] = 0.02 + 0.015 * torch.rand(blocks, hk, generator=gen, device=DEV)
        s["v_scale"] = 0.02 + 0.015 * torch.rand(blocks, hk, generator=gen, device=DEV)
    else:
        s["k_codes"], s["v_codes"] = _words(gen, blocks, hk, b, d // 8), _words(gen, blocks, hk, b // 8, d)
        s["k_scale"], s["v_scale"] = _scales(gen, blocks, hk, b), _scales(gen, blocks, hk, b)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["starts"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    s["most_new"], s["longest"] = max(new), max(lens)
    if case["op"] == "attend":
        s["q"] = normal(n, h, d).to(t)
        return s
    qkv = (normal(n, (h + 2 * hk) * d) * 1.5).to(t)
    s["q"] = qkv[:, :h * d].view(n, h, d)
    s["k"], s["v"] = qkv[:, h * d:(h + hk) * d].view(n, hk, d), qkv[:, (h + hk) * d:].view(n, hk, d)
    _turning(case, n, gen, s)
    s["positions"] = None
    if not case["implied"]:
        place = torch.cat([torch.arange(a - m, a) for a, m in zip(lens, new)]).to(DEV) + 1000 * (seed % 50)
        s["positions"] = (place if case["axes"] == 1 else torch.stack((place, place // 7, place % 7))).to(torch.int32).contiguous()
    return s


# --------------------------------------------------------------------------------------------------- run
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_turn(s):
    import dequant_matmul_qmv_amd as mxq
    return mxq.mxq_norm_rope(s["q"], s["k"], s["inv_freq"], s["positions"], s["q_weight"], s["k_weight"], eps=EPS,
                             axes=s["axes"], interleaved=s["case"]["interleaved"])


def _own_append(s):
    import dequant_matmul_qmv_amd as mxq
    kind = mxq.KvCache if s["case"]["bits"] == 8 else mxq.KvCache4
    cache = kind(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    q = mxq.mxq_rope_append(cache, s["q"], s["k"], s["v"], s["inv_freq"], s["table"], s["lens"],
                            None if s["case"]["new"] == "one" else s["starts"], s["q_weight"], s["k_weight"],
                            positions=s["positions"], axes=s["axes"], eps=EPS, interleaved=s["case"]["interleaved"])
    return q, cache.k, cache.v, cache.k_scale, cache.v_scale


def _own_attend(s):
    import dequant_matmul_qmv_amd as mxq
    cache = mxq.KvCache4(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    return mxq.mxq_attention(s["q"], cache, s["table"], s["lens"], None if s["case"]["new"] == "one" else s["starts"],
                             window=s["case"]["window"], return_lse=s["case"]["lse"])


_run_own = {"turn": _own_turn, "append": _own_append, "attend": _own_attend}


def _plain_rotated(s, x, weight, positions):
    """x normed and rotated, rounded once; every product and sum in 32 bits, angles and the mean of squares in 64."""
    case, rot = s["case"], s["case"]["rot"]
    y = x.float()
    if weight is not None:
        y = y * (1 / (x.double().square().mean(-1, keepdim=True) + EPS).sqrt()).float() * weight.float()
    if s["axes"] is None:
        angle = positions.double()[:, None] * s["inv_freq"].double()
    else:
        angle = positions[s["axes"].long()].T.double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((z, y[..., rot:]), -1).to(x.dtype)


def _plain_turn(s):
    return (_plain_rotated(s, s["q"], s["q_weight"], s["positions"]), _plain_rotated(s, s["k"], s["k_weight"], s["positions"]))


def _token_places(s, n):
    """For each new token: its sequence, its number among the sequence's new ones, its position."""
    starts, lens = s["starts"].long(), s["lens"].long()
    t = torch.arange(n, device=DEV)
    seq = torch.searchsorted(starts[1:], t, right=True)
    nth = t - starts[seq]
    return seq, nth, lens[seq] - (starts[seq + 1] - starts[seq]) + nth


def _plain_append(s):
    b = s["case"]["block"]
    seq, _, pos = _token_places(s, s["k"].shape[0])
    at = pos if s["positions"] is None else s["positions"]
    q, k = _plain_rotated(s, s["q"], s["q_weight"], at), _plain_rotated(s, s["k"], s["k_weight"], at)
    page, slot = s["table"][seq, pos // b].long(), pos % b
    if s["case"]["bits"] == 8:
        _plain_put8(s, k, page, slot)
    else:
        _plain_put4(s, k, page, slot)
    return q, s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]


def _plain_put8(s, k, page, slot):
    b = s["case"]["block"]
    first = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1])          # tokens that were there before
    part = torch.gather(s["table"], 1, (first // b).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    held = torch.where(part >= 0, first % b, 0)                              # ... of them in the block that is continued
    part = part.clamp(min=0)

    def put(codes, scale, x, by_token):
        x = x.float()
        fresh = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
        was = torch.zeros_like(scale)
        was[part] = torch.where(held[:, None] > 0, scale[part], 0.0)
        # quotients in 64 bits, rounded once: a 32-bit quotient is then the nearest one whatever the divider
        wide = torch.maximum(was, (fresh.double() / 127).float())
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEV)
        touched[page] = True
        scale.copy_(torch.where(touched[:, None], wide, scale))
        ratio = torch.where(wide > 0, was.double() / wide.double(), 0.0).float()[part][..., None, None]
        old = codes[part]
        keep = (torch.arange(b, device=DEV) < held[:, None])[:, None]
        keep = keep[..., None] if by_token else keep[:, :, None]
        codes[part] = torch.where(keep, (old.float() * ratio).round().to(torch.int8), old)
        inv = torch.where(wide > 0, 1 / wide.double(), 0.0).float().clamp(max=torch.finfo(torch.float32).max)
        c = (x * inv[page][..., None]).round().clamp(-127, 127).to(torch.int8)
        if by_token:
            codes[page, :, slot] = c
        else:
            codes[page, :, :, slot] = c

    put(s["k_codes"], s["k_scale"], k, True)
    put(s["v_codes"], s["v_scale"], s["v"], False)


def _plain_quantized4(x):
    """Codes int32 [tokens, kv heads, dim] and scale words int16 [tokens, kv heads]."""
    x = x.float()
    lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    step = (hi.double() - lo.double()) / 15                                  # a fifteenth of the range, zero within it,
    unit = torch.ldexp(torch.ones_like(step), (torch.frexp(step)[1] - 7).clamp(min=-20))
    scale = ((step / unit).ceil() * unit).clamp(max=4064.0)                  # up to the next number of 7 bits
    inv = torch.where(scale > 0, 1 / scale, 0.0).float()
    zero = (-lo * inv).round().clamp(max=15)
    codes = ((x * inv[..., None]).round() + zero[..., None]).clamp(0, 15).to(torch.int32)
    return codes, scale.to(torch.float16).view(torch.int16) | zero.to(torch.int16)


def _plain_put4(s, k, page, slot):
    n, hk, d = k.shape
    place = 4 * torch.arange(8, dtype=torch.int32, device=DEV)
    codes, scale = _plain_quantized4(k)
    s["k_codes"][page, :, slot] = (codes.view(n, hk, d // 8, 8) << place).sum(-1).to(torch.int32)
    s["k_scale"][page, :, slot] = scale
    codes, scale = _plain_quantized4(s["v"])
    s["v_scale"][page, :, slot] = scale
    # tokens that share words: their bits are cleared, then added (no two tokens have the same bits)
    mask, value = (15 << 4 * (slot % 8))[:, None, None].expand(n, hk, d), codes.long() << 4 * (slot % 8)[:, None, None]
    words = s["v_codes"].long() & 0xFFFFFFFF
    index = (page, slice(None), slot // 8)
    rows = page * (s["case"]["block"] // 8) + slot // 8                      # of [blocks * block / 8, kv heads, dim]
    flat = words.permute(0, 2, 1, 3).reshape(-1, hk, d)
    clear = torch.zeros_like(flat).index_add_(0, rows, mask)
    fresh = torch.zeros_like(flat).index_add_(0, rows, value)
    new = ((flat & ~clear) | fresh)[rows]
    s["v_codes"][index] = torch.where(new > 0x7FFFFFFF, new - (1 << 32), new).to(torch.int32)


def _plain_values(words, scales, token_words):
    """Values of words [..., tokens / 8, dim] (token_words) or [..., tokens, dim / 8]: [..., tokens, dim]."""
    place = 4 * torch.arange(8, dtype=torch.int32, device=DEV)
    if token_words:
        codes = ((words[..., None, :] >> place[:, None]) & 15).flatten(-3, -2)
    else:
        codes = ((words[..., None] >> place) & 15).flatten(-2)
    scale = (scales & 0x7FF0).view(torch.float16).float()[..., None]
    return (codes - (scales & 15).int()[..., None]).float() * scale


def _plain_attend(s):
    case = s["case"]
    hk, g, d, b = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], case["block"]
    n, most, width = case["seqs"], s["most_new"], -(-s["longest"] // case["block"])
    ids = s["table"][:, :width].long().clamp(min=0)
    k = _plain_values(s["k_codes"][ids], s["k_scale"][ids], False)           # [seqs, width, hk, b, d]
    v = _plain_values(s["v_codes"][ids], s["v_scale"][ids], True)
    k = k.permute(0, 2, 1, 3, 4).reshape(n, hk, width * b, d)
    v = v.permute(0, 2, 1, 3, 4).reshape(n, hk, width * b, d)
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
    seq, nth, _ = _token_places(s, s["q"].shape[0])
    out = y.permute(0, 3, 1, 2, 4).reshape(n, most, hk * g, d)[seq, nth].to(s["q"].dtype)
    if not case["lse"]:
        return out
    return out, (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(n, most, hk * g)[seq, nth]


_run_plain = {"turn": _plain_turn, "append": _plain_append, "attend": _plain_attend}


# -------------------------------------------------------------------------------------------------- work
def work(case):
    e, h, hk, d = 2, case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "turn":                              # q and k read and written; a square, a weight and a rotation a value
        n = case["tokens"] * (h + hk)
        return {"bytes": 2 * n * d * e + 4 * case["axes"] * case["tokens"] + 2 * case["rot"],
                "flops": n * (4 * d * case["norm"] + 3 * case["rot"])}
    lens, new = _lengths(case)
    if case["op"] == "append":                            # q read and written, k and v read, codes (and 4-bit scales) written
        n = sum(new)
        held = 1 if case["bits"] == 8 else 0.5 + 2 / d
        return {"bytes": n * d * (2 * h * e + 2 * hk * (e + held)) + (0 if case["implied"] else 4 * case["axes"] * n),
                "flops": n * ((h + hk) * (4 * d * case["norm"] + 3 * case["rot"]) + 6 * hk * d)}
    tokens = pairs = 0
    for length, n in zip(lens, new):
        w = case["window"] or length
        tokens += min(length, w + n - 1)
        full = max(0, min(n, length - w))                 # rows whose window is full
        rest = n - full                                   # the others see 1 + length - n .. tokens
        pairs += full * w + rest * (length - n) + rest * (rest + 1) // 2
    return {"bytes": 2 * tokens * hk * (d // 2 + 2) + 2 * sum(new) * h * d * e, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions, token by token or sequence by sequence, in 64 bits."""
    return {"turn": _exact_turn, "append": _exact_append, "attend": _exact_attend}[case["op"]](case, prepare(case, seed))


def _exact_rotated(case, s, x, weight, positions):
    """(a + ib) times e^(i angle) for each pair of the normed head."""
    half = case["rot"] // 2
    i = torch.arange(half, device=DEV)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, half + i)
    y = x.to(torch.float64).clone()
    if weight is not None:
        y /= ((y * y).sum(-1, keepdim=True) / case["dim"] + EPS) ** 0.5
        y *= weight.to(torch.float64)
    p = positions.to(torch.float64).reshape(-1, x.shape[0])
    which = torch.zeros(half, dtype=torch.int64, device=DEV) if s["axes"] is None else s["axes"].to(torch.int64)
    angle = p.T[:, which] * s["inv_freq"].to(torch.float64)
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_turn(case, s):
    return (_exact_rotated(case, s, s["q"], s["q_weight"], s["positions"]),
            _exact_rotated(case, s, s["k"], s["k_weight"], s["positions"]))


def _exact_append(case, s):
    """q, and the 8-bit scales; codes are whole numbers that the 32-bit rule alone defines, so they have no such value."""
    b, (lens, new) = case["block"], _lengths(case)
    at = s["positions"]
    if at is None:
        at = torch.cat([torch.arange(a - m, a) for a, m in zip(lens, new)]).to(DEV)
    q = _exact_rotated(case, s, s["q"], s["q_weight"], at)
    if case["bits"] == 4:
        return q, None, None, None, None
    k = _exact_rotated(case, s, s["k"], s["k_weight"], at).to(s["k"].dtype)  # keys have the storage type's rounding
    table, scales = s["table"].cpu(), []
    for name, x in (("k_scale", k), ("v_scale", s["v"])):
        peak = x.to(torch.float64).abs().amax(-1).cpu()
        scale = s[name].to(torch.float64).cpu()
        row0 = 0
        for i, (length, n) in enumerate(zip(lens, new)):
            begin = length - n
            for j in range(begin // b, -(-length // b)):
                lo, hi = max(begin, j * b), min(length, (j + 1) * b)
                got = peak[row0 + lo - begin:row0 + hi - begin].amax(0) / 127
                row = scale[table[i, j]]
                scale[table[i, j]] = torch.maximum(row, got) if j * b < begin else got
            row0 += n
        scales.append(scale)
    return q, None, None, scales[0], scales[1]


def _exact_values(words, scales, by_token):
    """Values [tokens, dim] of a sequence's pages of one head: words [pages, tokens, dim / 8], or [pages, tokens / 8, dim]."""
    parts = [(words >> (4 * j)).remainder(16).double() for j in range(8)]
    codes = torch.stack(parts, 2 if by_token else 3)
    codes = codes.flatten(0, 2) if by_token else codes.flatten(2, 3).flatten(0, 1)
    flat = scales.flatten().to(torch.int32)
    zero = (flat % 16).double()
    return (codes - zero[:, None]) * (flat - flat % 16).to(torch.int16).view(torch.float16).double()[:, None]


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
            k = _exact_values(s["k_codes"][ids, h], s["k_scale"][ids, h], False)[:length]
            v = _exact_values(s["v_codes"][ids, h], s["v_scale"][ids, h], True)[:length]
            for j in range(g):
                x = (q[:, h * g + j] @ k.T).masked_fill(hide, -math.inf)
                ls.append(x.logsumexp(-1))
                ys.append((x - ls[-1][:, None]).exp() @ v)
        out.append(torch.stack(ys, 1))
        lse.append(torch.stack(ls, 1))
        at += n
    return (torch.cat(out), torch.cat(lse)) if case["lse"] else torch.cat(out)
