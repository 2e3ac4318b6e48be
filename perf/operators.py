"""Cases for the 8-bit key/value cache: writing it, reading it back, attention over it, choosing blocks of it by a
cheap score, and attention over the chosen blocks.

A cache holds pages of 64 tokens.  K codes are [pages][hkv][64][d] and V codes [pages][hkv][d][64], where token
t = 16 j + 8 h + 2 c + e of a page stands at 16 c + 4 j + 2 h + e; codes are float8 e4m3 or int8.  Each (page, kv head)
has a K and a V scale, a power of two ([pages][hkv][2] fp32), and the floor and ceiling of its K channels' minimum and
maximum ([pages][hkv][2][d] int8, in units of the K scale for int8 and of four K scales for e4m3).  A page table
[sequences][columns] and lengths [sequences], which count the tokens of the call, say where a sequence lies; the rows of
a call are the newest tokens of each sequence, packed, with prefix sums `cu` (None: one row for each sequence).
"""
import math
import random

import torch

own = False

BLOCK = 64
LARGEST = {"e4m3": 448.0, "int8": 127.0}
INF = float("inf")


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a serving batch writes its new token for each sequence
        dict(name="append_step", op="append", n=256, lo=64, hi=8192, new=1, fresh=False, hkv=8, d=128, fmt="e4m3", mix=1),
        # a packed micro-batch of about 32K prompt tokens (256 to 32K each) is written after its attention
        dict(name="append_prompts", op="append", n=7, lo=256, hi=32768, new=0, fresh=True, hkv=8, d=128, fmt="int8", mix=2),
        # the same kind of prompts is read back as bf16, to attend to what the cache holds
        dict(name="read_prompts", op="read", n=7, lo=256, hi=32768, new=0, hkv=8, d=128, fmt="e4m3", mix=3),
        # a 128K sequence leaves the cache for host memory or another rank
        dict(name="read_seq128k", op="read", n=1, lo=131072, hi=131072, new=0, hkv=8, d=128, fmt="int8", mix=4),
        # the smallest call: four short documents, one new token each; launch latency counts
        dict(name="attend_tiny", op="attend", n=4, lo=64, hi=512, new=1, hq=4, hkv=4, d=64, fmt="e4m3", mix=5),
        # an ordinary decoding step: 64 sequences of very different lengths
        dict(name="attend_batch", op="attend", n=64, lo=256, hi=32768, new=1, hq=32, hkv=8, d=128, fmt="e4m3", mix=6),
        # up to five drafted tokens for each sequence are checked in one pass
        dict(name="attend_draft", op="attend", n=16, lo=1024, hi=32768, new=5, hq=32, hkv=8, d=128, fmt="int8", mix=7),
        # one token over the longest context, 2M tokens
        dict(name="attend_seq2m", op="attend", n=1, lo=2097152, hi=2097152, new=1, hq=32, hkv=8, d=128, fmt="int8", mix=8),
        # blocks chosen for a batch of long sequences
        dict(name="select_batch", op="select", n=16, lo=8192, hi=131072, new=1, hq=32, hkv=8, d=128, fmt="e4m3", count=64, mix=9),
        # blocks chosen among the 32,768 of a 2M-token context
        dict(name="select_seq2m", op="select", n=1, lo=2097152, hi=2097152, new=1, hq=32, hkv=8, d=128, fmt="int8", count=256, mix=10),
        # attention over 32 chosen blocks of each sequence of a batch
        dict(name="sparse_batch", op="sparse", n=64, lo=4096, hi=32768, new=1, hq=32, hkv=8, d=128, fmt="int8", count=32, mix=11),
        # attention over 256 chosen blocks of a 2M-token context
        dict(name="sparse_seq2m", op="sparse", n=1, lo=2097152, hi=2097152, new=1, hq=32, hkv=8, d=128, fmt="e4m3", count=256, mix=12),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "select", "sparse"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    longest = _spread(rng, 100, 1 << 21)
    room = (1 << 31) // (hkv * d)  # padded tokens: no more than the largest listed case holds
    if op in ("append", "read"):
        room //= 8
    longest = min(longest, room)
    n = max(1, min(_spread(rng, 1, 256), room // longest))
    lo = max(1, _spread(rng, 1, longest))
    new = 1 if op == "sparse" or rng.random() < 0.5 else rng.randint(2, 6)
    case = dict(op=op, n=n, lo=lo, hi=longest, new=new, hkv=hkv, d=d, fmt=rng.choice(["e4m3", "int8"]), mix=rng.randrange(1 << 20))
    if op == "append":
        case["fresh"] = rng.random() < 0.5
        if case["fresh"]:
            case["new"] = 0
    elif op == "read":
        case["new"] = 0
    else:
        case["hq"] = hkv * group
    if op in ("select", "sparse"):
        case["count"] = min(_spread(rng, 3, 512), room // (BLOCK * n))
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


def work(case):
    lens, new = shape(case)
    hkv, d, rows = case["hkv"], case["d"], sum(new)
    if case["op"] in ("append", "read"):
        touched = sum((l - 1) // BLOCK - (l - m) // BLOCK + 1 for l, m in zip(lens, new))
        sides = touched * hkv * (8 + (2 * d if case["op"] == "append" else 0))
        return {"bytes": rows * hkv * d * 2 * (2 + 1) + sides, "flops": rows * hkv * d * 4}
    hq = case["hq"]
    if case["op"] == "select":
        blocks = sum((l - 1) // BLOCK + 1 for l in lens)
        pairs = sum(m * ((l - 1) // BLOCK + 1) for l, m in zip(lens, new))
        return {"bytes": blocks * hkv * (2 * d + 4) + rows * hq * d * 2 + rows * hkv * case["count"] * 4, "flops": pairs * hkv * d * 4}
    if case["op"] == "attend":
        keys = sum(lens)
        pairs = sum(m * l for l, m in zip(lens, new))
    else:
        keys = pairs = sum(min(l, case["count"] * BLOCK) for l in lens)
    blocks = keys / BLOCK
    return {"bytes": keys * hkv * d * 2 + blocks * hkv * 8 + rows * hq * (d * 4 + 4), "flops": pairs * hq * d * 4}


# ---------------------------------------------------------------- the inputs

def _pow2(e):
    """2^e as fp32, -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _normal(shape_, std, g, dtype=torch.bfloat16):
    return (torch.randn(shape_, generator=g, device="cuda") * std).to(dtype)


def _codes(shape_, fmt, g):
    """Codes of normally distributed values whose largest magnitude fills most of the type's range."""
    x = torch.empty(shape_, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // max(1, x[0].numel()))
    for a in range(0, shape_[0], step):
        part = x[a:a + step]
        y = torch.randn(part.shape, generator=g, device="cuda") * (LARGEST[fmt] / 4.2)
        y = y.clamp_(-LARGEST[fmt], LARGEST[fmt])
        part.copy_((y.round_().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)).view(torch.uint8))
    return x


def _bounds(k, fmt):
    lo = torch.empty((k.shape[0], k.shape[1], 2, k.shape[3]), dtype=torch.int8, device="cuda")
    step = max(1, (1 << 27) // max(1, k[0].numel()))
    for a in range(0, k.shape[0], step):
        x = k[a:a + step]
        x = x.view(torch.int8).float() if fmt == "int8" else x.view(torch.float8_e4m3fn).float() / 4
        lo[a:a + step, :, 0] = x.amin(2).floor().to(torch.int8)
        lo[a:a + step, :, 1] = x.amax(2).ceil().to(torch.int8)
    return lo


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens, new = shape(case)
    n, hkv, d, fmt, op = case["n"], case["hkv"], case["d"], case["fmt"], case["op"]
    columns = [(l + BLOCK - 1) // BLOCK for l in lens]
    pages, width = sum(columns), max(columns)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)  # pages are handed out in no order
    table = torch.zeros((n, width), dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(columns):
        table[i, :c] = order[at:at + c]
        at += c
    s = dict(op=op, fmt=fmt, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), rows=sum(new), most=max(new), d=d, hkv=hkv)
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    s["cu"] = None if case["new"] == 1 else torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["k"], s["v"] = _codes((pages, hkv, BLOCK, d), fmt, g), _codes((pages, hkv, d, BLOCK), fmt, g)
    s["bounds"] = _bounds(s["k"], fmt)
    # scales of values of order one; some heads and blocks are a few times larger
    top = math.log2(LARGEST[fmt])
    s["scales"] = _pow2(torch.randint(0, 3, (pages, hkv, 2), generator=g, device="cuda") + round(1.5 - top))
    if op == "append":
        s["k_new"], s["v_new"] = _normal((s["rows"], hkv, d), 1.0, g), _normal((s["rows"], hkv, d), 1.0, g)
        s["k_new"][:, :, :: d // 4] *= 4  # a few channels of K are larger than the others, as in trained models
    if op in ("attend", "select", "sparse"):
        s["q"] = _normal((s["rows"], case["hq"], d), 1.0, g)
        s["scale"] = 1.0 / math.sqrt(d)
    if op in ("select", "sparse"):
        s["count"] = case["count"]
        s["first"], s["last"] = 1, min(2, case["count"] - 1)
    if op == "sparse":  # one token for each sequence: distinct blocks, ascending, -1 behind
        count = case["count"]
        lists = torch.full((n, hkv, count), -1, dtype=torch.int32, device="cuda")
        for i, c in enumerate(columns):
            m = min(c, count)
            pick = torch.rand((hkv, c), generator=g, device="cuda")
            pick[:, c - 1] = 2
            lists[i, :, :m] = pick.topk(m, dim=1).indices.sort(dim=1).values.to(torch.int32)
        s["blocks"] = lists
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


def _typed(x, fmt):
    return x.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)


def _in_order(v):
    """V codes [..., d, 64] with the tokens of a page in their order."""
    return v.unflatten(-1, (4, 4, 2, 2)).movedim(-4, -2).flatten(-4)


def _as_stored(v):
    return v.unflatten(-1, (4, 2, 4, 2)).movedim(-2, -4).flatten(-4)


def _power(x, most):
    """The exponent of the smallest power of two, 2^-126 at least, that `most` times reaches x."""
    m, e = torch.frexp(x)
    f, b = math.frexp(most)
    return torch.where(x > 0, e - b + (m > f), -126).clamp(min=-126)


def _plain_append(s):
    fmt, hkv, d, T, n = s["fmt"], s["hkv"], s["d"], s["rows"], s["lens"].numel()
    most = LARGEST[fmt]
    lens = s["lens"].long()
    cu = torch.arange(n + 1, device="cuda") if s["cu"] is None else s["cu"].long()
    # a slot for every block that the call may touch: sequence i has cu[i+1]/64 - cu[i]/64 + 2 of them
    slots = torch.arange(T // BLOCK + 2 * n, device="cuda")
    start = cu[:-1] // BLOCK + 2 * torch.arange(n, device="cuda")
    seq = torch.searchsorted(start, slots, right=True) - 1
    p0 = lens[seq] - (cu[seq + 1] - cu[seq])
    block = p0 // BLOCK + slots - start[seq]
    held = block * BLOCK < lens[seq]
    seq, p0, block = seq[held], p0[held], block[held]
    page = s["table"][seq, block].long()
    pos = block[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    is_new = (pos >= p0[:, None]) & (pos < lens[seq][:, None])
    row = (cu[seq][:, None] + pos - p0[:, None]).clamp(0, T - 1)
    fresh = block * BLOCK >= p0

    def write(x, old, old_scale):
        """New codes (as values) and scales; x [m][64][hkv][d] rows, old [m][hkv][64][d] code values."""
        x = torch.where(is_new[:, :, None, None], x.float(), 0.0)
        need = _pow2(_power(x.abs().amax((1, 3)), most))
        scale = torch.where(fresh[:, None], need, torch.maximum(need, old_scale))
        old = torch.where(fresh[:, None, None, None], 0.0, old * (old_scale / scale)[:, :, None, None])
        y = torch.where(is_new[:, None, :, None], x.transpose(1, 2) / scale[:, :, None, None], old)
        return y.round() if fmt == "int8" else y.to(torch.float8_e4m3fn).float(), scale, x

    stored = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    scale0 = s["scales"][page]
    y, k_scale, x = write(s["k_new"][row], _typed(s["k"][page], fmt).float(), scale0[..., 0])
    s["k"][page] = y.to(stored).view(torch.uint8)
    unit = (k_scale if fmt == "int8" else 4 * k_scale)[..., None]
    low = torch.where(is_new[:, :, None, None], x, INF).amin(1)
    high = torch.where(is_new[:, :, None, None], x, -INF).amax(1)
    old = s["bounds"][page].float() * (scale0[..., 0] / k_scale)[..., None, None]
    low = torch.minimum((low / unit).floor(), torch.where(fresh[:, None, None], INF, old[:, :, 0].floor()))
    high = torch.maximum((high / unit).ceil(), torch.where(fresh[:, None, None], -INF, old[:, :, 1].ceil()))
    s["bounds"][page] = torch.stack((low, high), 2).to(torch.int8)
    y, v_scale, _ = write(s["v_new"][row], _in_order(_typed(s["v"][page], fmt).float()).transpose(2, 3), scale0[..., 1])
    s["v"][page] = _as_stored(y.transpose(2, 3)).to(stored).view(torch.uint8)
    s["scales"][page] = torch.stack((k_scale, v_scale), 2)


def _written(s):
    return {"k": _typed(s["k"], s["fmt"]), "v": _typed(s["v"], s["fmt"]), "scales": s["scales"], "bounds": s["bounds"]}


def _plain_read(s):
    seq, pos = _rows(s)
    page, inside = s["table"][seq, pos // BLOCK].long(), pos % BLOCK
    j, h, c, e = inside // 16, inside // 8 % 2, inside // 2 % 4, inside % 2
    scale = s["scales"][page]
    k = _typed(s["k"], s["fmt"])[page, :, inside].float() * scale[..., :1]
    v = _typed(s["v"], s["fmt"])[page, :, :, 16 * c + 4 * j + 2 * h + e].float() * scale[..., 1:]
    return {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


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
    scale = s["scales"][page]
    k = _typed(s["k"][page], s["fmt"]).float().mul_(scale[..., 0, None, None]).transpose(1, 2).reshape(n, hkv, width * BLOCK, d)
    v = _in_order(_typed(s["v"][page], s["fmt"]).float().mul_(scale[..., 1, None, None]))
    v = v.permute(0, 2, 1, 4, 3).reshape(n, hkv, width * BLOCK, d)
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


def _plain_select(s):
    hkv, d, count = s["hkv"], s["d"], s["count"]
    T, hq = s["q"].shape[:2]
    seq, pos = _rows(s)
    q = s["q"].float().reshape(T, hkv, hq // hkv, d)
    c = (q * _pow2(-_power(q.abs().amax((2, 3)), 127.0))[:, :, None, None]).round().double()
    up, down = c.clamp(min=0).sum(2), c.clamp(max=0).sum(2)
    page = s["table"].long()
    bounds = s["bounds"][page].double()
    low, high = (bounds[..., i, :].permute(0, 2, 3, 1)[seq] for i in (0, 1))
    total = (down[:, :, None] @ low + up[:, :, None] @ high).squeeze(2)  # whole numbers, exact in 64 bits
    score = total.float() * s["scales"][page][..., 0].transpose(1, 2)[seq]
    b = torch.arange(page.shape[1], device="cuda")
    have = (pos // BLOCK + 1)[:, None, None]
    score = torch.where(b < have, score, -INF)
    kept = ((b < s["first"]) | (b >= have - s["last"])) & (b < have)
    order = score.sort(dim=-1, descending=True, stable=True).indices
    rank = kept.expand_as(score).gather(-1, order).float() + (b < have).expand_as(score).gather(-1, order)
    order = order.gather(-1, rank.sort(dim=-1, descending=True, stable=True).indices)[..., :count]
    order = torch.where(order < have, order, page.shape[1]).sort(dim=-1).values
    found = torch.full((T, hkv, count), -1, dtype=torch.int32, device="cuda")
    found[..., :order.shape[-1]] = torch.where(order < page.shape[1], order, -1)
    return found


def _plain_sparse(s):
    hkv, d = s["hkv"], s["d"]
    T, hq = s["q"].shape[:2]
    seq, pos = _rows(s)
    b = s["blocks"].long()
    count = b.shape[-1]
    page = s["table"][seq[:, None, None], b.clamp(min=0)].long()
    head = torch.arange(hkv, device="cuda")[None, :, None]
    scale = s["scales"][page, head]
    k = (_typed(s["k"][page, head], s["fmt"]).float() * scale[..., 0, None, None]).reshape(T, hkv, count * BLOCK, d)
    v = _in_order(_typed(s["v"][page, head], s["fmt"]).float() * scale[..., 1, None, None])
    v = v.transpose(3, 4).reshape(T, hkv, count * BLOCK, d)
    key = b[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
    seen = ((b[..., None] >= 0) & (key <= pos[:, None, None, None])).reshape(T, hkv, 1, count * BLOCK)
    q = s["q"].float().reshape(T, hkv, hq // hkv, d)
    o, lse = _softmax((q @ k.transpose(2, 3)) * s["scale"], seen, v)
    return {"o": o.reshape(T, hq, d).to(torch.bfloat16), "lse": lse.reshape(T, hq).t().contiguous()}


# ---------------------------------------------------------------- one pass

def _own(s):
    import packed_varlen_attention_aware_gb300 as hdp

    fmt = hdp.HDP_CACHE_INT8 if s["fmt"] == "int8" else hdp.HDP_CACHE_E4M3
    cache = hdp.KVCache(s["k"], s["v"], s["scales"], s["bounds"], fmt)
    if s["op"] == "append":
        hdp.cache_append(cache, s["table"], s["lens"], s["k_new"], s["v_new"], cu=s["cu"])
        return _written(s)
    if s["op"] == "read":
        k, v = hdp.cache_read(cache, s["table"], s["lens"], s["rows"], cu=s["cu"])
        return {"k": k, "v": v}
    if s["op"] == "select":
        return hdp.cache_select(cache, s["table"], s["lens"], s["q"], s["count"], cu=s["cu"], keep_first=s["first"], keep_last=s["last"])
    o, lse = hdp.cache_attention(cache, s["table"], s["lens"], s["q"], cu=s["cu"], blocks=s.get("blocks"), scale=s["scale"])
    return {"o": o, "lse": lse}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "append":
        _plain_append(s)
        return _written(s)
    return {"read": _plain_read, "attend": _plain_attend, "select": _plain_select, "sparse": _plain_sparse}[s["op"]](s)


# ---------------------------------------------------------------- in 64 bits, from the definition

def _two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _value(codes, fmt):
    """Code bytes as float64, by the meaning of their bits."""
    x = codes.to(torch.int64)
    if fmt == "int8":
        return torch.where(x > 127, x - 256, x).double()
    e, f = x // 8 % 16, (x % 8).double()
    size = torch.where(e > 0, (1 + f / 8) * _two_to(e - 7), f / 8 * 2.0 ** -6)
    return torch.where(x > 127, -size, size)


def _rounded(x, fmt):
    if fmt == "int8":
        return torch.round(x)
    step = _two_to(torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return torch.round(x / step) * step


def _smallest(top, most):
    """The smallest power of two, 2^-126 at least, with top <= most times it."""
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / most)).clamp(min=-126)
    e = torch.where(top <= most * _two_to(e - 1), e - 1, e)
    e = torch.where(top > most * _two_to(e), e + 1, e)
    return _two_to(e.clamp(min=-126))


TOKEN = [16 * c + 4 * j + 2 * h + e for j in range(4) for h in range(2) for c in range(4) for e in range(2)]


def _sequence(s, i, count, head=slice(None)):
    """Dequantised K and V [hkv][keys][d] of the first `count` blocks of sequence i."""
    page = s["table"][i, :count].long()
    k = _value(s["k"][page][:, head], s["fmt"]) * s["scales"][page][:, head, 0, None, None].double()
    v = _value(s["v"][page][:, head], s["fmt"])[..., TOKEN] * s["scales"][page][:, head, 1, None, None].double()
    return k.transpose(0, 1).flatten(1, 2), v.permute(1, 0, 3, 2).flatten(1, 2)


def _exact_append(s, case, lens, new):
    fmt, most = s["fmt"], LARGEST[s["fmt"]]
    kv = {"k": _value(s["k"], fmt), "v": _value(s["v"], fmt)}
    scales, bounds = s["scales"].double(), s["bounds"].double()
    row = 0
    for i, (l, m) in enumerate(zip(lens, new)):
        for b in range((l - m) // BLOCK, (l - 1) // BLOCK + 1):
            p = int(s["table"][i, b])
            a, z = max(b * BLOCK, l - m), min(l, b * BLOCK + BLOCK)
            inside = slice(a - b * BLOCK, z - b * BLOCK)
            for which, name in enumerate("kv"):
                x = s[name + "_new"][row + a - (l - m):row + z - (l - m)].double().transpose(0, 1)  # [hkv][rows][d]
                scale = _smallest(x.abs().amax((1, 2)), most)
                codes = kv[name][p] if name == "k" else kv[name][p][..., TOKEN].transpose(1, 2)
                if a > b * BLOCK:
                    scale = torch.maximum(scale, scales[p, :, which])
                    codes = _rounded(codes * (scales[p, :, which] / scale)[:, None, None], fmt)
                else:
                    codes = torch.zeros_like(codes)
                codes[:, inside] = _rounded(x / scale[:, None, None], fmt)
                if name == "k":
                    kv[name][p] = codes
                    unit = (scale if fmt == "int8" else 4 * scale)[:, None]
                    low, high = torch.floor(x.amin(1) / unit), torch.ceil(x.amax(1) / unit)
                    if a > b * BLOCK:
                        ratio = (scales[p, :, 0] / scale)[:, None]
                        low = torch.minimum(low, torch.floor(bounds[p, :, 0] * ratio))
                        high = torch.maximum(high, torch.ceil(bounds[p, :, 1] * ratio))
                    bounds[p, :, 0], bounds[p, :, 1] = low, high
                else:
                    kv[name][p][..., TOKEN] = codes.transpose(1, 2)
                scales[p, :, which] = scale
        row += m
    whole = (lambda x: x.to(torch.int64)) if fmt == "int8" else (lambda x: x)
    return {"k": whole(kv["k"]), "v": whole(kv["v"]), "scales": scales, "bounds": bounds.to(torch.int64)}


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = shape(case)
    op, hkv, d = case["op"], case["hkv"], case["d"]
    if op == "append":
        return _exact_append(s, case, lens, new)
    if op == "read":
        got = [_sequence(s, i, (l + BLOCK - 1) // BLOCK) for i, l in enumerate(lens)]
        return {n: torch.cat([x[w][:, l - m:l].transpose(0, 1) for x, l, m in zip(got, lens, new)]) for w, n in enumerate("kv")}
    hq = case["hq"]
    g = hq // hkv
    if op == "select":
        found = torch.full((s["rows"], hkv, s["count"]), -1, dtype=torch.int64)
        scales, bounds, table, q = (s[x].double().cpu() for x in ("scales", "bounds", "table", "q"))
        row = 0
        for i, (l, m) in enumerate(zip(lens, new)):
            for r in range(m):
                have = (l - m + r) // BLOCK + 1
                page = table[i, :have].long()
                for h in range(hkv):
                    x = q[row, h * g:(h + 1) * g]
                    c = torch.round(x / _smallest(x.abs().amax(), 127.0))
                    total = torch.maximum(c[:, None], torch.zeros(())).sum(0) * bounds[page, h, 1] + torch.minimum(c[:, None], torch.zeros(())).sum(0) * bounds[page, h, 0]
                    score = total.sum(-1).float().double() * scales[page, h, 0]
                    score[:s["first"]] = INF
                    score[max(0, have - s["last"]):] = INF
                    pick = sorted(score.sort(descending=True, stable=True).indices[:s["count"]].tolist())
                    found[row, h, :len(pick)] = torch.tensor(pick)
                row += 1
        return found
    o = torch.zeros((s["rows"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((hq, s["rows"]), -INF, dtype=torch.float64, device="cuda")
    row = 0
    for i, (l, m) in enumerate(zip(lens, new)):
        for h in range(hkv):
            k, v = (x[0] for x in _sequence(s, i, (l + BLOCK - 1) // BLOCK, slice(h, h + 1)))
            for r in range(m):
                keys = slice(0, l - m + r + 1)
                if op == "sparse":
                    b = s["blocks"][row + r, h].long()
                    keys = (b[b >= 0][:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten()
                    keys = keys[keys <= l - m + r]
                x = k[keys] @ s["q"][row + r, h * g:(h + 1) * g].double().t() * s["scale"]
                lse[h * g:(h + 1) * g, row + r] = torch.logsumexp(x, 0)
                o[row + r, h * g:(h + 1) * g] = torch.softmax(x, 0).t() @ v[keys]
        row += m
    return {"o": o, "lse": lse}
