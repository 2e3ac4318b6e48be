"""Cases for serving and training around the packed attention: block tables and slot maps made on the GPU from the
requests' lengths, rotary positions and their gradient, and a key/value cache held in 4 bits (writing it, reading it
back, attention over it).

The pool of pages is a stack of free pages: free int32 [pages], count int32 [1], its top at count - 1.  A sequence of l
tokens holds ceil(l / 64) pages, listed in its row of the page table.

A 4-bit cache holds pages of 64 tokens: codes of 4 bits (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two in
a byte, the first in its low half.  K codes are [pages][hkv][64][d / 2], where channel 32 g + 8 c + 2 b + e of a token
stands in byte (d / 8) c + 4 g + b, half e.  V codes are [pages][hkv][d / 16][512], where channel 16 i + 8 h + r of
token 16 s + 8 p + 2 c + e stands in byte 64 r + 16 c + 8 h + 2 s + p of row i, half e.  Scales are powers of two, held
as their exponent plus 127 in a byte (255: NaN): one for each token, kv head and 32 channels of K, and one for each
token and kv head of V, [pages][hkv][d / 32 + 1][64], V's in the last row, token 8 j + r at place 8 r + j.
"""
import math
import random

import torch

own = False

BLOCK = 64
INF = float("inf")
MOST = 6.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TURN = 2 * math.pi


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a decoding step of a serving batch: pages for the sequences that enter a new block, the new tokens' slots; then the step is taken back
        dict(name="tables_step", op="tables", n=256, lo=64, hi=8192, new=1, mix=1),
        # prompts are admitted and, finished, give their pages back
        dict(name="tables_prompts", op="tables", n=64, lo=256, hi=32768, new=0, mix=2),
        # rotary positions of the new tokens of a decoding step, some of them far into long contexts
        dict(name="rotary_step", op="rotary", n=256, lo=64, hi=2097152, new=1, hq=32, hkv=8, d=128, rot=128, type="bf16", pairs="halves", fused=True, back=False, mix=3),
        # q and k of a packed micro-batch of about 32K tokens, where the projection left them
        dict(name="rotary_batch", op="rotary", n=8, lo=256, hi=32768, new=0, hq=32, hkv=8, d=128, rot=128, type="bf16", pairs="halves", fused=True, back=False, mix=4),
        # the gradients of q and k of a 128K sequence, half of each head turned
        dict(name="rotary_seq128k_back", op="rotary", n=1, lo=131072, hi=131072, new=0, hq=32, hkv=8, d=128, rot=64, type="bf16", pairs="neighbours", fused=False, back=True, mix=5),
        # one decoding step writes its new token for each sequence; the rows come back as the cache holds them
        dict(name="write_step", op="write", n=256, lo=64, hi=8192, new=1, hkv=8, d=128, mix=6),
        # a packed micro-batch of prompts is written, and read back to attend to what the cache holds
        dict(name="write_prompts", op="write", n=7, lo=256, hi=32768, new=0, hkv=8, d=128, mix=7),
        # prompts that are in the cache already are read back as bf16
        dict(name="read_prompts", op="read", n=7, lo=256, hi=32768, new=0, hkv=8, d=128, mix=8),
        # a 128K sequence leaves the cache for host memory or another rank
        dict(name="read_seq128k", op="read", n=1, lo=131072, hi=131072, new=0, hkv=8, d=128, mix=9),
        # the smallest call: four short documents, one new token each; launch latency counts
        dict(name="attend_tiny", op="attend", n=4, lo=64, hi=512, new=1, hq=4, hkv=4, d=64, mix=10),
        # an ordinary decoding step: 64 sequences of very different lengths
        dict(name="attend_batch", op="attend", n=64, lo=256, hi=32768, new=1, hq=32, hkv=8, d=128, mix=11),
        # one token over the longest context, 2M tokens
        dict(name="attend_seq2m", op="attend", n=1, lo=2097152, hi=2097152, new=1, hq=32, hkv=8, d=128, mix=12),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rotary", "rotary", "write", "read", "attend", "attend", "attend"])
    mix = rng.randrange(1 << 20)
    longest = _spread(rng, 100, 1 << 21)
    if op == "tables":
        n = max(1, min(_spread(rng, 1, 1024), (1 << 21) // longest))
        return dict(op=op, n=n, lo=max(1, _spread(rng, 1, longest)), hi=longest, new=rng.choice([0, 1, rng.randint(2, 6), rng.randint(7, 700)]), mix=mix)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    if op == "rotary":
        step = rng.random() < 0.5
        room = (1 << 29) // ((hq + hkv) * d)  # rows: no more than the largest listed case has
        if not step:
            longest = min(longest, room)
        n = max(1, min(_spread(rng, 1, 512 if step else 256), room if step else room // longest))
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
        return dict(op=op, n=n, lo=max(1, _spread(rng, 1, longest)), hi=longest, new=rng.randint(1, 5) if step else 0, hq=hq, hkv=hkv, d=d, rot=rot, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    pairs=rng.choice(["halves", "neighbours"]), fused=rng.random() < 0.5, back=rng.random() < 0.4, mix=mix)
    room = (1 << 31) // (hkv * d) // (8 if op != "attend" else 1)  # padded tokens: no more than the largest listed case holds
    longest = min(longest, room)
    n = max(1, min(_spread(rng, 1, 256), room // longest))
    case = dict(op=op, n=n, lo=max(1, _spread(rng, 1, longest)), hi=longest, new=1 if rng.random() < 0.5 else rng.randint(2, 6), hkv=hkv, d=d, mix=mix)
    if op == "read" or (op == "write" and rng.random() < 0.5):
        case["new"] = 0
    if op == "attend":
        case["hq"] = hq
    return case


def shape(case):
    """Lengths of the sequences, and how many newest tokens each has in the call (new = 0: all of them)."""
    r = random.Random(case["mix"])
    lens = [_spread(r, case["lo"], case["hi"]) for _ in range(case["n"])]
    if case["new"] == 0:
        return lens, list(lens)
    if case["new"] == 1:
        return lens, [1] * len(lens)
    return lens, [min(l, r.randint(1, case["new"])) for l in lens]


def _blocks(l):
    return (l + BLOCK - 1) // BLOCK


def work(case):
    lens, new = shape(case)
    rows = sum(new)
    if case["op"] == "tables":
        moved = sum(_blocks(l) - _blocks(l - m) for l, m in zip(lens, new))
        return {"bytes": case["n"] * 4 * 6 + moved * 4 * 4 + rows * 16, "flops": 0}
    d = case["d"]
    if case["op"] == "rotary":
        heads = case["hq"] + case["hkv"]
        return {"bytes": rows * (heads * d * (4 if case["type"] == "fp32" else 2) * 2 + 4) + case["rot"] * 4, "flops": rows * heads * case["rot"] * 3}
    hkv = case["hkv"]
    held = d + d // 32 + 1  # bytes of a token and kv head
    if case["op"] == "write":
        return {"bytes": rows * hkv * (d * 4 + held + d * 4), "flops": rows * hkv * d * 4}
    if case["op"] == "read":
        return {"bytes": rows * hkv * (held + d * 4), "flops": rows * hkv * d * 2}
    keys, pairs, hq = sum(lens), sum(m * l for l, m in zip(lens, new)), case["hq"]
    return {"bytes": keys * hkv * held + rows * hq * (d * 4 + 4), "flops": pairs * hq * d * 4}


# ---------------------------------------------------------------- the inputs

def _on(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _normal(shape_, std, g, dtype=torch.bfloat16):
    return (torch.randn(shape_, generator=g, device="cuda") * std).to(dtype)


def _cu(case, new):
    if case["new"] == 1:
        return None
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    return _on(cu)


def _frequencies(rot, base=500000.0):
    """Angle of one position for each pair, in radians; contexts of eight times the length trained on: the slow pairs
    turn eight times slower, the fast ones as trained, with a ramp between them."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** -(i / rot)
    turns = 8192 * f / TURN  # over the length trained on
    keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
    return (f * (keep + (1 - keep) / 8)).to("cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens, new = shape(case)
    n, op, rows = case["n"], case["op"], sum(new)
    s = dict(op=op, rows=rows, most=max(new), lens=_on(lens), cu=_cu(case, new))
    if op == "rotary":
        hq, hkv, d, t = case["hq"], case["hkv"], case["d"], TYPES[case["type"]]
        if case["fused"]:  # q, k and v of a token side by side
            x = _normal((rows, hq + 2 * hkv, d), 1.0, g, t)
            s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hkv]
        else:
            s["q"], s["k"] = _normal((rows, hq, d), 1.0, g, t), _normal((rows, hkv, d), 1.0, g, t)
        seq, pos = _rows(s)
        # documents of a micro-batch begin at 0, requests go on where they are; a few are moved on
        s["positions"] = (pos + torch.randint(0, 3, (n,), generator=g, device="cuda")[seq] * 1000).to(torch.int32)
        s["freqs"], s["factor"] = _frequencies(case["rot"]), 0.1 * math.log(8) + 1
        s["neighbours"], s["back"] = case["pairs"] == "neighbours", case["back"]
        return s
    columns = [_blocks(l) for l in lens]
    pages, width = sum(columns), max(columns)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)  # pages are handed out in no order
    table = torch.zeros((n, width), dtype=torch.int32, device="cuda")
    held = [_blocks(l - m) for l, m in zip(lens, new)] if op == "tables" else columns
    at = 0
    for i, c in enumerate(held):
        table[i, :c] = order[at:at + c]
        at += c
    s["table"] = table
    if op == "tables":
        s["before"] = _on([l - m for l, m in zip(lens, new)])
        s["held"], s["free"], s["count"] = _on(held), torch.zeros(pages, dtype=torch.int32, device="cuda"), _on([pages - at])
        s["free"][:pages - at] = order[at:]
        return s
    hkv, d = case["hkv"], case["d"]
    s["d"], s["hkv"] = d, hkv
    s["codes_k"] = torch.randint(0, 256, (pages, hkv, BLOCK, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    s["codes_v"] = torch.randint(0, 256, (pages, hkv, d // 16, 512), generator=g, device="cuda", dtype=torch.uint8)
    # scales of values of order one; some tokens and groups of channels are a few times larger
    s["scales"] = torch.randint(124, 128, (pages, hkv, d // 32 + 1, BLOCK), generator=g, device="cuda", dtype=torch.uint8)
    if op == "write":
        s["k"], s["v"] = _normal((rows, hkv, d), 1.0, g), _normal((rows, hkv, d), 1.0, g)
        s["k"][:, :, :: d // 4] *= 4  # a few channels of K are larger than the others, as in trained models
    if op == "attend":
        s["q"] = _normal((rows, case["hq"], d), 0.5, g)
        s["scale"] = 1.0 / math.sqrt(d)
    return s


# ---------------------------------------------------------------- plain forms

def _rows(s):
    """(sequence, position) of every row of the call."""
    t = torch.arange(s["rows"], device="cuda")
    if s["cu"] is None:
        return t, s["lens"].long() - 1
    cu = s["cu"].long()
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return seq, s["lens"].long()[seq] - cu[seq + 1] + t


def _plain_assign(s, lens):
    """Pages for the blocks of `lens`: what a sequence no longer needs goes back on the stack, the last sequence's last
    block first; then each sequence takes what it lacks from the top, in order, as long as there is enough."""
    have, want = s["held"].long(), (lens.long() + BLOCK - 1) // BLOCK
    back, lack = (have - want).clamp(min=0), (want - have).clamp(min=0)
    col = torch.arange(s["table"].shape[1], device="cuda")
    end = s["count"].long() + back.sum()
    place = end - 1 - ((back.cumsum(0) - back)[:, None] + col - want[:, None])
    given = (col >= want[:, None]) & (col < have[:, None])
    free = torch.cat((s["free"], s["free"][:1]))
    free.scatter_(0, torch.where(given, place, free.numel() - 1).flatten(), s["table"].flatten())
    before = lack.cumsum(0) - lack
    fits = before + lack <= end
    lack = torch.where(fits, lack, 0)
    place = end - 1 - (before[:, None] + col - have[:, None])
    taken = (col >= have[:, None]) & (col < (have + lack)[:, None])
    s["table"].copy_(torch.where(taken, free[place.clamp(0, free.numel() - 1)], s["table"]))
    s["free"].copy_(free[:-1])
    s["held"].copy_(torch.where(back > 0, want, have + lack))
    s["count"].copy_(end - lack.sum())


def _plain_tables(s):
    _plain_assign(s, s["lens"])
    seq, pos = _rows(s)
    slot = s["table"][seq, pos // BLOCK].long() * BLOCK + pos % BLOCK
    _plain_assign(s, s["before"])
    return {"sequence": seq.to(torch.int32), "position": pos.to(torch.int32), "slot": slot, **_pool(s)}


def _pool(s):
    return {"table": s["table"], "held": s["held"], "free": s["free"], "count": s["count"]}


def _plain_turn(x, cos, sin, neighbours):
    """Pairs (x1, x2) of the first channels of a head, turned: (x1 cos - x2 sin, x2 cos + x1 sin)."""
    rot = 2 * cos.shape[-1]
    y = x.float()
    cos, sin = cos[:, None], sin[:, None]
    if neighbours:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _plain_rotary(s):
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    if s["back"]:
        sin = -sin
    return {x: _plain_turn(s[x], cos, sin, s["neighbours"]) for x in "qk"}


SIZES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values(codes):
    """Bytes [..., m] as the 2 m values of their codes, the low half's first."""
    size = torch.tensor(SIZES, device="cuda")
    one = torch.cat((size, -size))
    both = torch.stack((one.repeat(16), one.repeat_interleave(16)), -1)
    return both[codes.int()].flatten(-2)


def _nearest(y):
    """Code of y, |y| <= 6: the nearest value, of two equally near ones the one with the even code."""
    a = y.abs()
    c = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return c + 8 * (y < 0).byte()


def _bytes_of(codes):
    return codes[..., 0::2] | codes[..., 1::2] << 4


def _pow2(e):
    """2^e as fp32 of an exponent -127 <= e <= 127."""
    return torch.ldexp(torch.ones((), device="cuda"), e.float())


def _exponent(top):
    """The exponent of the smallest power of two, 2^-126 at least, that six times reaches `top`."""
    m, e = torch.frexp(top)  # 6 = 0.75 * 2^3
    return torch.where(top > 0, e - 3 + (m > 0.75), -126).clamp(min=-126)


def _k_stored(x):
    """Channels of K [..., d] in the order of their halves of bytes."""
    return x.unflatten(-1, (-1, 4, 8)).transpose(-3, -2).flatten(-3)


def _k_channels(x):
    return x.unflatten(-1, (4, -1, 8)).transpose(-3, -2).flatten(-3)


def _v_tokens(x):
    """Values of V codes [..., d / 16, 1024] as [..., 64, d]: from (i, r, c, h, s, p, e) to (s, p, c, e), (i, h, r)."""
    x = x.unflatten(-1, (8, 4, 2, 4, 2, 2))
    a = x.dim() - 7
    lead = list(range(a))
    return x.permute(*lead, a + 4, a + 5, a + 2, a + 6, a, a + 3, a + 1).flatten(-3).flatten(-5, -2)


def _in_order(x):
    """Places of a page's scales [..., 64] as tokens, and the way back."""
    return x.unflatten(-1, (8, 8)).transpose(-1, -2).flatten(-2)


def _plain_write(s):
    hkv, d = s["hkv"], s["d"]
    seq, pos = _rows(s)
    page, at = s["table"][seq, pos // BLOCK].long(), pos % BLOCK
    k, v = s["k"].float(), s["v"].float()
    ek, ev = _exponent(k.unflatten(-1, (-1, 32)).abs().amax(-1)), _exponent(v.abs().amax(-1))
    place = at % 8 * 8 + at // 8
    s["scales"][page, :, :, place] = torch.cat((ek, ev[..., None]), -1).add(127).to(torch.uint8)
    code = _nearest((k.unflatten(-1, (-1, 32)) / _pow2(ek)[..., None]).flatten(-2))
    s["codes_k"][page, :, at] = _bytes_of(_k_stored(code))
    code = _nearest(v / _pow2(ev)[..., None])
    # V's bytes hold two tokens: the even ones' halves, then the odd ones'
    ch = torch.arange(d, device="cuda")
    row = ch // 16
    byte = ch % 8 * 64 + ch // 8 % 2 * 8 + (at // 2 % 4 * 16 + at // 16 * 2 + at // 8 % 2)[:, None]
    head = torch.arange(hkv, device="cuda")[:, None]
    where = (page[:, None, None], head, row, byte[:, None])
    for half in (0, 1):
        mine = (at % 2 == half)[:, None, None]
        old = s["codes_v"][where]
        new = torch.where(mine, old & (15 << 4 - 4 * half) | code << 4 * half, old)
        # rows of the other half write what their byte holds; where their partner is a row too, its new byte
        partner = torch.arange(s["rows"], device="cuda") + (1 if half else -1)
        inside = partner.clamp(0, s["rows"] - 1)
        paired = (partner == inside) & (seq[inside] == seq) & (pos[inside] // 2 == pos // 2)
        s["codes_v"][where] = torch.where(mine | ~paired[:, None, None], new, new[inside])
    return {**_plain_read(s), "scales": s["scales"].view(torch.float8_e8m0fnu)}


def _plain_read(s):
    seq, pos = _rows(s)
    page, at = s["table"][seq, pos // BLOCK].long(), pos % BLOCK
    hkv, d = s["hkv"], s["d"]
    scale = _pow2(s["scales"][page, :, :, at % 8 * 8 + at // 8].int() - 127)
    k = _k_channels(_values(s["codes_k"][page, :, at])).unflatten(-1, (-1, 32)) * scale[..., :-1, None]
    ch = torch.arange(d, device="cuda")
    byte = ch % 8 * 64 + ch // 8 % 2 * 8 + (at // 2 % 4 * 16 + at // 16 * 2 + at // 8 % 2)[:, None]
    code = s["codes_v"][page[:, None, None], torch.arange(hkv, device="cuda")[:, None], ch // 16, byte[:, None]]
    code = code >> (at % 2 * 4).to(torch.uint8)[:, None, None] & 15
    v = _values(code[..., None])[..., 0::2].flatten(-2) * scale[..., -1:]
    return {"k": k.flatten(-2).to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _softmax(scores, seen, values):
    """(o, lse) of scores [..., r, keys] over the keys that are seen, values [..., keys, d]."""
    scores = scores.masked_fill(~seen, -INF)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -INF, 0.0, top)
    p = (scores - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ values) / torch.where(total == 0, 1.0, total)
    return o, (top + total.log()).squeeze(-1)


def _plain_attend(s):
    hkv, d = s["hkv"], s["d"]
    n, width = s["table"].shape
    T, hq = s["q"].shape[:2]
    g, m = hq // hkv, s["most"]
    page = s["table"].long()
    scale = _pow2(_in_order(s["scales"][page]).int() - 127)  # [n][width][hkv][d / 32 + 1][64]
    k = _k_channels(_values(s["codes_k"][page])).unflatten(-1, (-1, 32)).mul_(scale[..., :-1, :].transpose(-1, -2)[..., None])
    k = k.flatten(-2).transpose(1, 2).reshape(n, hkv, width * BLOCK, d)
    v = _v_tokens(_values(s["codes_v"][page])).mul_(scale[..., -1, :, None])
    v = v.transpose(1, 2).reshape(n, hkv, width * BLOCK, d)
    cu = torch.arange(n + 1, device="cuda") if s["cu"] is None else s["cu"].long()
    r = torch.arange(m, device="cuda")
    row = (cu[:-1, None] + r).clamp(max=T - 1)
    pos = s["lens"].long()[:, None] - (cu[1:] - cu[:-1])[:, None] + r
    q = s["q"][row].float().reshape(n, m, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, m * g, d)
    seen = torch.arange(width * BLOCK, device="cuda") <= pos[:, :, None]
    seen = seen[:, None, :, None].expand(n, 1, m, g, -1).reshape(n, 1, m * g, -1)
    o, lse = _softmax((q @ k.transpose(2, 3)) * s["scale"], seen, v)
    seq = _rows(s)[0]
    mine = torch.arange(T, device="cuda") - cu[seq]
    o = o.reshape(n, hkv, m, g, d)[seq, :, mine].reshape(T, hq, d)
    lse = lse.reshape(n, hkv, m, g)[seq, :, mine].reshape(T, hq)
    return {"o": o.to(torch.bfloat16), "lse": lse.t().contiguous()}


# ---------------------------------------------------------------- one pass

def _own(s):
    import packed_varlen_attention_aware_gb300 as hdp

    op = s["op"]
    if op == "tables":
        pool = hdp.PagePool(s["free"], s["count"])
        hdp.cache_assign(pool, s["table"], s["held"], s["lens"])
        seq, pos, slot = hdp.cache_rows(s["lens"], s["rows"], cu=s["cu"], page_table=s["table"], num_pages=pool.num_pages)
        hdp.cache_assign(pool, s["table"], s["held"], s["before"])
        return {"sequence": seq, "position": pos, "slot": slot, **_pool(s)}
    if op == "rotary":
        turn = hdp.rotary_backward if s["back"] else hdp.rotary
        q, k = turn(s["q"], s["k"], s["positions"], s["freqs"], neighbours=s["neighbours"], factor=s["factor"])
        return {"q": q, "k": k}
    cache = hdp.KVCache4(s["codes_k"], s["codes_v"], s["scales"])
    if op == "attend":
        o, lse = hdp.cache_attention(cache, s["table"], s["lens"], s["q"], cu=s["cu"], scale=s["scale"])
        return {"o": o, "lse": lse}
    if op == "write":
        hdp.cache_append(cache, s["table"], s["lens"], s["k"], s["v"], cu=s["cu"])
    k, v = hdp.cache_read(cache, s["table"], s["lens"], s["rows"], cu=s["cu"])
    return {"k": k, "v": v, "scales": s["scales"].view(torch.float8_e8m0fnu)} if op == "write" else {"k": k, "v": v}


def run(s):
    if own:
        return _own(s)
    return {"tables": _plain_tables, "rotary": _plain_rotary, "write": _plain_write, "read": _plain_read, "attend": _plain_attend}[s["op"]](s)


# ---------------------------------------------------------------- in 64 bits, from the definition

def _code_values(codes):
    """The two values of each byte, as float64, by the meaning of their bits."""
    x = codes.long()
    out = []
    for c in (x & 15, x >> 4):
        e, m = (c >> 1 & 3).double(), (c & 1).double()
        size = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1), m / 2)
        out.append(torch.where(c > 7, -size, size))
    return torch.stack(out, -1)


def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale_values(s, page):
    """[..., planes, 64 tokens] as float64."""
    t = torch.arange(BLOCK, device="cuda")
    return _two_to(s["scales"][page].long()[..., t % 8 * 8 + t // 8] - 127)


def _sequence(s, i, count, h):
    """Dequantised K and V [keys][d] of kv head h in the first `count` blocks of sequence i."""
    d = s["d"]
    page = s["table"][i, :count].long()
    scale = _scale_values(s, page)[:, h]
    ch = torch.arange(d, device="cuda")
    k = _code_values(s["codes_k"][page, h])  # [blocks][64][d / 2][2]
    k = k[:, :, d // 8 * (ch % 32 // 8) + 4 * (ch // 32) + ch % 8 // 2, ch % 2] * scale[:, ch // 32].transpose(1, 2)
    t = torch.arange(BLOCK, device="cuda")[:, None]
    byte = 64 * (ch % 8) + 16 * (t // 2 % 4) + 8 * (ch // 8 % 2) + 2 * (t // 16) + t // 8 % 2
    v = _code_values(s["codes_v"][page, h])  # [blocks][d / 16][512][2]
    v = v[:, ch // 16, byte, t % 2] * scale[:, -1, :, None]
    return k.flatten(0, 1), v.flatten(0, 1)


def _round4(y):
    """To the nearest of the 4-bit values, ties to the even one: steps of 1/2 up to 2, of 1 up to 4, of 2 above."""
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return torch.sign(y) * torch.round(a / step) * step


def _smallest(top):
    """The smallest power of two, 2^-126 at least, with top <= 6 times it."""
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / MOST)).clamp(min=-126)
    e = torch.where(top <= MOST * _two_to(e - 1), e - 1, e)
    e = torch.where(top > MOST * _two_to(e), e + 1, e)
    return _two_to(e.clamp(min=-126))


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    lens, new = shape(case)
    d = case["d"]
    if case["op"] == "rotary":
        rot, found = case["rot"], {}
        angle = s["positions"].double()[:, None, None] * s["freqs"] * (-1 if s["back"] else 1)
        z = torch.polar(torch.full_like(angle, s["factor"]), angle)
        for name in "qk":
            x = s[name].double()
            y = x.clone()
            first, second = (slice(0, rot, 2), slice(1, rot, 2)) if s["neighbours"] else (slice(0, rot // 2), slice(rot // 2, rot))
            w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z
            y[..., first], y[..., second] = w.real, w.imag
            found[name] = y
        return found
    hkv = case["hkv"]
    if case["op"] == "write":
        k, v = s["k"].double().unflatten(-1, (-1, 32)), s["v"].double()
        sk, sv = _smallest(k.abs().amax(-1, keepdim=True)), _smallest(v.abs().amax(-1, keepdim=True))
        return {"k": (_round4(k / sk) * sk).flatten(-2), "v": _round4(v / sv) * sv}
    if case["op"] == "read":
        out = [torch.empty((s["rows"], hkv, d), dtype=torch.float64, device="cuda") for _ in "kv"]
        row = 0
        for i, (l, m) in enumerate(zip(lens, new)):
            for h in range(hkv):
                for to, x in zip(out, _sequence(s, i, _blocks(l), h)):
                    to[row:row + m, h] = x[l - m:l]
            row += m
        return dict(zip("kv", out))
    hq = case["hq"]
    g = hq // hkv
    o = torch.zeros((s["rows"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((hq, s["rows"]), -INF, dtype=torch.float64, device="cuda")
    row = 0
    for i, (l, m) in enumerate(zip(lens, new)):
        for h in range(hkv):
            k, v = _sequence(s, i, _blocks(l), h)
            for r in range(m):
                end = l - m + r + 1
                x = k[:end] @ s["q"][row + r, h * g:(h + 1) * g].double().t() * s["scale"]
                lse[h * g:(h + 1) * g, row + r] = torch.logsumexp(x, 0)
                o[row + r, h * g:(h + 1) * g] = torch.softmax(x, 0).t() @ v[:end]
        row += m
    return {"o": o, "lse": lse}
