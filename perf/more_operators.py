"""Workloads of appending with the position rotation, of attention through a sliding
window with first tokens that stay visible, and of attention of a batch that shares
a prefix.

Four operators, named by a case's "op":

  rotate  new tokens' keys, rotated by their positions, and values into a paged
          cache (quantised to 8 bits by their head's scale, or kept in 16), and
          the queries rotated beside them
  window  attention of each sequence's newest tokens over its pages: a token sees
          the `window` newest tokens up to itself and the first `sinks`
  prompt  the same over packed prompts of different lengths
  shared  attention over pages, groups of sequences sharing their first tokens

A case gives sizes; the sequences' lengths follow from it alone (`_lengths`), the
values from the seed.  With `own` false the operators are computed in their plain
form (elementary torch operations), with `own` true by this repository's entry
points.
"""
import math
import random

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# largest value, fraction bits, exponent of the smallest normal
_FP8 = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}


def listed():
    base = dict(batch=1, q_min=1, q_max=1, kv_min=0, kv_max=0, lens=1, heads=32, kv_heads=8,
                dim=128, page=16, layout="NHD", dtype="bf16", cache="same")

    def case(name, op, **over):
        return {"name": name, "op": op, **base, **over}
    return [
        # one decode step of a serving batch: a token of each of 64 requests into an
        # 8-bit cache, its query rotated beside it (latency)
        case("rotate_step", "rotate", batch=64, kv_min=500, kv_max=8192, cache="e4m3", page=64,
             rotary=128, style="halves", base=500000.0),
        # prompts of about 13k tokens in all into an 8-bit cache
        case("rotate_prompts", "rotate", batch=12, q_min=37, q_max=4096, kv_min=37, kv_max=6000,
             cache="e4m3", page=16, layout="HND", rotary=128, style="halves", base=10000.0),
        # a 16-bit cache with pages of an odd size, half of each small head rotated by
        # pairs, chunks far into long contexts
        case("rotate_partial", "rotate", batch=9, q_min=101, q_max=2001, kv_min=2001,
             kv_max=100001, dtype="f16", heads=16, kv_heads=4, dim=64, page=24, rotary=32,
             style="pairs", base=10000.0),
        # a few requests decoding through a short window: the smallest attention call
        case("window_few", "window", batch=4, kv_min=100, kv_max=2000, page=16, window=512, sinks=4),
        # the decode batch at contexts up to 32k through a window of 4,096
        case("window_batch", "window", batch=64, kv_min=500, kv_max=32768, page=64, layout="HND",
             window=4096, sinks=4),
        # chunked prefill over an 8-bit cache
        case("window_chunk", "window", batch=8, q_min=200, q_max=1024, kv_min=1024, kv_max=16384,
             cache="e4m3", page=32, dtype="f16", window=2000, sinks=16),
        # short prompts of odd lengths, small heads, a narrow window
        case("window_prompts", "prompt", batch=24, q_min=1, q_max=2500, lens=5, heads=12, kv_heads=4,
             dim=64, dtype="f16", window=333, sinks=1),
        # one whole prompt of 16,384 tokens through a window of 4,096
        case("window_prompt_long", "prompt", batch=1, q_min=16384, q_max=16384, window=4096, sinks=0),
        # a few requests behind one system prompt that ends inside a page
        case("shared_few", "shared", batch=5, kv_min=10, kv_max=200, page=16, groups=1,
             shared_min=1500, shared_max=1500, loose=0),
        # a decode batch behind one long shared document
        case("shared_batch", "shared", batch=64, kv_min=30, kv_max=1000, page=64, layout="HND",
             groups=1, shared_min=16384, shared_max=16384, loose=0),
        # an 8-bit cache, eight query heads to a kv head, several prompts shared by their groups
        case("shared_groups", "shared", batch=96, kv_min=100, kv_max=3000, heads=64, cache="e4m3",
             page=64, groups=5, shared_min=2000, shared_max=16000, loose=3),
        # questions of different lengths about one document, all at once
        case("shared_questions", "shared", batch=16, q_min=30, q_max=400, kv_min=30, kv_max=400,
             page=32, dtype="f16", groups=1, shared_min=16000, shared_max=16000, loose=0),
    ]


_MOST_PAIRS = 70_000_000 * 32      # row-key pairs of all heads of the largest listed case
_MOST_ROWS = 13_000 * 48           # head rows of the largest append
_MOST_KEYS = 400_000 * 8           # head keys of the largest


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("rotate", "window", "window", "prompt", "shared", "shared"))
        dim = rng.choice((64, 128, 128))
        kv_heads = rng.choice((1, 2, 4, 8))
        group = rng.choice((1, 2, 3, 4, 5, 8, 16))
        c = dict(op=op, batch=_log(rng, 1, 96), q_min=1, q_max=1, kv_min=0, kv_max=0,
                 lens=rng.randrange(1, 1 << 20), heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                 page=rng.choice((16, 16, 32, 64, 64, 128, 24, 20)),
                 layout=rng.choice(("NHD", "HND")), dtype=rng.choice(("bf16", "f16")),
                 cache=rng.choice(("same", "same", "e4m3", "e5m2")))
        if op == "prompt":
            c["q_max"] = _log(rng, 20, 16384)
            c["q_min"] = rng.choice((c["q_max"], max(1, c["q_max"] // 9)))
        else:
            c["kv_max"] = _log(rng, 40, 4000 if op == "shared" else 32768)
            c["kv_min"] = max(1, c["kv_max"] // rng.choice((1, 4, 30)))
            if rng.random() < 0.5:
                c["q_max"] = min(c["kv_max"], _log(rng, 2, 2048))
                c["q_min"] = rng.choice((c["q_max"], max(1, c["q_max"] // 5)))
        if op == "rotate":
            c.update(rotary=rng.choice((dim, dim, dim // 2, dim // 4)), style=rng.choice(("halves", "pairs")),
                     base=rng.choice((10000.0, 500000.0)))
        elif op == "shared":
            groups, loose = rng.choice((1, 1, 2, 4, 7)), rng.choice((0, 0, 2))
            c["batch"] = max(c["batch"], 2 * groups + loose)
            c.update(groups=groups, shared_max=_log(rng, 100, 16384), loose=loose)
            c["shared_min"] = max(1, c["shared_max"] // rng.choice((1, 3)))
        else:
            c.update(window=_log(rng, 16, 4096), sinks=rng.choice((0, 1, 4, 64)))
        rows, pairs, keys = _counts(c)
        if op == "rotate":
            if not 64 <= rows * (c["heads"] + 2 * kv_heads) <= _MOST_ROWS:
                continue
        elif pairs * c["heads"] > _MOST_PAIRS or keys * kv_heads > _MOST_KEYS:
            continue
        return c


def _lengths(case):
    """(new tokens, tokens in all) of each sequence; with a shared prefix the second
    counts it, too."""
    r = random.Random(case["lens"])
    q = [_log(r, case["q_min"], case["q_max"]) for _ in range(case["batch"])]
    q[0] = case["q_max"]
    if case["op"] == "prompt":
        return q, list(q)
    kv = [_log(r, max(case["kv_min"], 1), case["kv_max"]) for _ in range(case["batch"])]
    kv[-1] = case["kv_max"]
    kv = [max(a, b) for a, b in zip(q, kv)]
    if case["op"] == "shared":
        cu, shared = _groups(case)
        for g, n in enumerate(shared):
            for b in range(cu[g], cu[g + 1]):
                kv[b] += n
    return q, kv


def _groups(case):
    """Sequences cu[g] .. cu[g + 1] - 1 share their first shared[g] tokens; the last
    `loose` sequences share nothing."""
    r = random.Random(case["lens"] + 1)
    n = case["batch"] - case["loose"]
    cuts = sorted(r.sample(range(1, n), case["groups"] - 1)) if case["groups"] > 1 else []
    shared = [_log(r, case["shared_min"], case["shared_max"]) for _ in range(case["groups"])]
    shared[0] = case["shared_max"]
    return [0] + cuts + [n], shared


def _seen(case, first, last):
    """The keys that rows at positions first .. last of a sequence see between them, as
    (tokens from the start, first of the rest): 0 .. a - 1 and b .. last."""
    if "window" not in case:
        return 0, 0
    b = max(0, first - case["window"] + 1)
    return min(case["sinks"], b), b


def _counts(case):
    """Rows, row-key pairs that are seen, and keys that are seen by a row at least."""
    q_lens, kv_lens = _lengths(case)
    pairs = keys = 0
    for n, total in zip(q_lens, kv_lens):
        off = total - n
        a, b = _seen(case, off, total - 1)
        keys += a + total - b
        if "window" in case:
            W, S = case["window"], case["sinks"]
            # row p sees min(p + 1, W) of the window and min(S, max(0, p + 1 - W)) sinks
            pairs += sum(min(p + 1, W) + min(S, max(0, p + 1 - W)) for p in range(off, total))
        else:
            pairs += n * total - n * (n - 1) // 2
    if case["op"] == "shared":
        cu, shared = _groups(case)
        keys -= sum((cu[g + 1] - cu[g] - 1) * n for g, n in enumerate(shared))
    return sum(q_lens), pairs, keys


def _round_fp8(x, kind):
    """Float64 values on the grid of an 8-bit format: nearest, ties to even, saturating."""
    largest, bits, low = _FP8[kind]
    x = x.clamp(-largest, largest)
    step = torch.exp2((torch.frexp(x).exponent - 1).clamp(min=low).double() - bits)
    return (torch.round(x / step) * step).clamp(-largest, largest)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    dt, B, H, D = _TYPES[c["dtype"]], c["batch"], c["kv_heads"], c["dim"]
    q_lens, kv_lens = _lengths(c)
    T = sum(q_lens)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32).cuda()

    def cumulative(lens):
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        return ints(cu)
    # q, k and v of the new tokens come out of one projection
    qkv = normal(T, c["heads"] + 2 * H, D)
    s = {"case": c, "cu": cumulative(q_lens), "q_lens": q_lens, "kv_lens": kv_lens, "max_q": max(q_lens),
         "tokens": T, "q": qkv[:, : c["heads"]], "k": qkv[:, c["heads"]: c["heads"] + H],
         "v": qkv[:, c["heads"] + H:], "scale": 1.0 / math.sqrt(D), "scale_k": None, "scale_v": None}
    if c["op"] == "prompt":
        return s
    page = c["page"]
    table, pages = [], 0
    leader, shared_of = list(range(B)), [0] * B     # whose pages hold a sequence's first tokens, how many
    if c["op"] == "shared":
        cu, shared = _groups(c)
        s["cu_shared"], s["shared_lens"] = ints(cu), ints(shared)
        for i, n in enumerate(shared):
            for b in range(cu[i], cu[i + 1]):
                leader[b], shared_of[b] = cu[i], n
    s["leader"], s["shared_of"] = leader, shared_of
    for b, (n, total) in enumerate(zip(q_lens, kv_lens)):
        slots = -(-total // page)
        row = [-1] * slots
        kept = range(slots)
        if c["op"] == "window":
            # pages behind every new token's window have been given back, but for the first tokens'
            a, lo = _seen(c, total - n, total - 1)
            kept = [x for x in kept if x * page < a or (x + 1) * page > lo]
        if c["op"] == "shared" and leader[b] != b:
            whole = shared_of[b] // page
            row[:whole] = table[leader[b]][:whole]
            kept = range(whole, slots)
        for x in kept:
            row[x] = pages
            pages += 1
        table.append(row)
    pages += 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    width = max(len(r) for r in table)
    t = torch.tensor([r + [-1] * (width - len(r)) for r in table], dtype=torch.int32)
    t = torch.where(t >= 0, order[t.clamp(min=0).long()], t)
    s["table"], s["lens"] = t.cuda(), ints(kv_lens)
    shape = (pages, page, H, D) if c["layout"] == "NHD" else (pages, H, page, D)
    s["pages_k"], s["pages_v"] = normal(*shape), normal(*shape)
    if c["op"] == "shared":
        # a prompt that ends inside a page: each sequence goes on in its own copy of that page
        for b in range(B):
            slot, rest = divmod(shared_of[b], page)
            if leader[b] != b and rest:
                for x in (s["pages_k"], s["pages_v"]):
                    x = x if c["layout"] == "NHD" else x.transpose(1, 2)
                    x[int(t[b, slot]), :rest] = x[int(t[leader[b], slot]), :rest]
    if c["cache"] != "same":
        largest = _FP8[c["cache"]][0]
        # what a calibration gives: the largest magnitude seen of each head
        amax = 3.5 + 2.5 * torch.rand(2, H, generator=g, device="cuda")
        s["scale_k"], s["scale_v"] = (amax[0] / largest).contiguous(), (amax[1] / largest).contiguous()
        for n, sc in (("pages_k", s["scale_k"]), ("pages_v", s["scale_v"])):
            by = sc.view(1, 1, H, 1) if c["layout"] == "NHD" else sc.view(1, H, 1, 1)
            s[n] = (s[n].float() / by).clamp(-largest, largest).to(_TYPES[c["cache"]])
    if c["op"] == "rotate":
        i = torch.arange(0, c["rotary"], 2, device="cuda", dtype=torch.float32)
        s["inv_freq"] = c["base"] ** (-i / c["rotary"])
    return s


def _rotated(c, x, pos, inv_freq):
    """Rows x (tokens, heads, dim) turned by their positions, float64 (far positions'
    angles, values next to a border between two codes)."""
    angle = pos.double()[:, None] * inv_freq.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    x, r = x.double(), c["rotary"]
    y = x.clone()
    if c["style"] == "halves":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y[..., : r // 2], y[..., r // 2: r] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _put(s, pages, x, scale, page, place):
    c = s["case"]
    if c["cache"] != "same":
        x = _round_fp8(x.double() / scale.double().view(1, -1, 1), c["cache"])
        x = x.float().to(_TYPES[c["cache"]]).view(torch.uint8)
    else:
        x = x.to(_TYPES[c["dtype"]])
    to = pages.view(torch.uint8) if c["cache"] != "same" else pages
    if c["layout"] == "NHD":
        to[page, place] = x
    else:
        to.permute(0, 2, 1, 3)[page, place] = x
    return pages


def _append(s):
    c, cu = s["case"], s["cu"].long()
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = s["lens"].long()[b] - (cu[b + 1] - t)
    page, place = s["table"].long()[b, pos // c["page"]], pos % c["page"]
    q = _rotated(c, s["q"], pos, s["inv_freq"]).to(_TYPES[c["dtype"]])
    k = _rotated(c, s["k"], pos, s["inv_freq"])
    return (q, _put(s, s["pages_k"], k, s["scale_k"], page, place),
            _put(s, s["pages_v"], s["v"].float(), s["scale_v"], page, place))


def _keys(s, b, at, pages, packed, scale):
    """Float32 (kv_heads, tokens, dim) of tokens `at` of sequence b."""
    c = s["case"]
    if c["op"] == "prompt":
        return packed[sum(s["q_lens"][:b]) + at].float().permute(1, 0, 2)
    table = s["table"].long()
    slot, place = at // c["page"], at % c["page"]
    page = table[b][slot]
    if c["op"] == "shared":
        page = torch.where(at < s["shared_of"][b], table[s["leader"][b]][slot], page)
    x = pages.view(torch.uint8) if c["cache"] != "same" else pages
    x = x[page, place] if c["layout"] == "NHD" else x.permute(0, 2, 1, 3)[page, place]
    x = (x.view(_TYPES[c["cache"]]) if c["cache"] != "same" else x).float().permute(1, 0, 2)
    return x if scale is None else x * scale.view(-1, 1, 1)


def _attend(s):
    """Plain attention, sequence by sequence and at most 1,024 rows at a time, float32."""
    c = s["case"]
    H, D, Hq = c["kv_heads"], c["dim"], c["heads"]
    G, t = Hq // H, 0
    out = torch.empty(s["tokens"], Hq, D, dtype=_TYPES[c["dtype"]], device="cuda")
    lse = torch.empty(s["tokens"], Hq, device="cuda")
    for b, (n, total) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        for i in range(0, n, 1024):
            m = min(1024, n - i)
            first, last = total - n + i, total - n + i + m - 1
            a, lo = _seen(c, first, last)
            at = torch.arange(lo, last + 1, device="cuda")
            if a:
                at = torch.cat([torch.arange(a, device="cuda"), at])
            pos = torch.arange(first, last + 1, device="cuda")[:, None]
            seen = at <= pos
            if "window" in c:
                seen &= (at > pos - c["window"]) | (at < c["sinks"])
            k = _keys(s, b, at, s.get("pages_k"), s["k"], s["scale_k"])
            v = _keys(s, b, at, s.get("pages_v"), s["v"], s["scale_v"])
            q = s["q"][t + i: t + i + m].float().view(m, H, G, D).permute(1, 2, 0, 3).reshape(H, G * m, D)
            x = torch.matmul(q * s["scale"], k.transpose(1, 2)).view(H, G, m, -1)
            x.masked_fill_(~seen, -math.inf)
            top = x.amax(-1, keepdim=True)
            x.sub_(top).exp_()
            z = x.sum(-1, keepdim=True)
            o = torch.matmul(x.view(H, G * m, -1), v).view(H, G, m, D) / z
            out[t + i: t + i + m] = o.permute(2, 0, 1, 3).reshape(m, Hq, D).to(out.dtype)
            lse[t + i: t + i + m] = (top + z.log()).squeeze(-1).permute(2, 0, 1).reshape(m, Hq)
        t += n
    return out, lse


def run(s):
    c = s["case"]
    if not own:
        return _append(s) if c["op"] == "rotate" else _attend(s)
    import sparse_attention_serving_sfa_gb300 as sfa
    if c["op"] == "prompt":
        return sfa.varlen_attention(s["q"], s["k"], s["v"], s["cu"], s["cu"], s["scale"], return_lse=True,
                                    max_q_len=s["max_q"], window=c["window"], sinks=c["sinks"])
    cache = dict(kv_layout=c["layout"], scale_k=s["scale_k"], scale_v=s["scale_v"])
    if c["op"] == "rotate":
        q = sfa.paged_append_rotated(s["k"], s["v"], s["cu"], s["pages_k"], s["pages_v"], s["table"],
                                     s["lens"], s["inv_freq"], q=s["q"], interleaved=c["style"] == "pairs",
                                     **cache)
        return q, s["pages_k"], s["pages_v"]
    if c["op"] == "window":
        return sfa.paged_attention(s["q"], s["pages_k"], s["pages_v"], s["table"], s["lens"], s["cu"],
                                   s["scale"], return_lse=True, max_q_len=s["max_q"], window=c["window"],
                                   sinks=c["sinks"], **cache)
    return sfa.shared_prefix_attention(s["q"], s["pages_k"], s["pages_v"], s["table"], s["lens"], s["cu"],
                                       s["cu_shared"], s["shared_lens"], s["scale"], return_lse=True,
                                       max_q_len=s["max_q"], **cache)


def work(case):
    """Each new row, and each cached token that a row sees, read or written once."""
    T, pairs, keys = _counts(case)
    D, Hq, H, B = case["dim"], case["heads"], case["kv_heads"], case["batch"]
    cached = 2 if case["cache"] == "same" else 1
    lists = 4 * (2 * B + 1)
    if case["op"] == "rotate":
        table = 4 * sum(-(-n // case["page"]) for n in _lengths(case)[0])
        return {"bytes": 4 * T * Hq * D + 2 * T * H * D * (2 + cached) + table + lists + 2 * case["rotary"],
                "flops": 3 * T * (Hq + H) * case["rotary"]}
    kv_bytes = 2 * keys * H * D * (2 if case["op"] == "prompt" else cached)
    table = 0 if case["op"] == "prompt" else 4 * (keys // case["page"])
    if case["op"] == "shared":
        lists += 4 * (2 * case["groups"] + 1)
    return {"bytes": 4 * T * Hq * D + 4 * T * Hq + kv_bytes + table + lists, "flops": 4 * D * Hq * pairs}


def _grid(kind):
    """The 8-bit format's non-negative values in order, decoded from their codes by its definition."""
    e5 = kind == "e5m2"
    bits, bias = (2, 15) if e5 else (3, 7)
    values = []
    for code in range(128):
        e, f = code >> bits, code & ((1 << bits) - 1)
        if (e5 and e == 31) or (not e5 and code == 127):
            break
        values.append(f * 2.0 ** (1 - bias - bits) if e == 0 else (1 + f / (1 << bits)) * 2.0 ** (e - bias))
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def exact(case, seed):
    s = prepare(case, seed)
    q_lens, kv_lens = _lengths(case)
    D, Hq, H = case["dim"], case["heads"], case["kv_heads"]
    first = [sum(q_lens[:b]) for b in range(len(q_lens))]
    hnd = case["layout"] == "HND"

    def slots(b, t):
        """Flat (page * page size + place) numbers of tokens t of sequence b."""
        size = case["page"]
        return s["table"][b].long()[torch.div(t, size, rounding_mode="floor")] * size + t % size

    if case["op"] == "rotate":
        r = case["rotary"]
        turned_q = torch.empty(sum(q_lens), Hq, D, dtype=torch.float64, device="cuda")
        got = [s["pages_k"].double(), s["pages_v"].double()]
        for b, n in enumerate(q_lens):
            t = torch.arange(kv_lens[b] - n, kv_lens[b], device="cuda")
            # turning a pair of coordinates = multiplying a complex number by exp(i angle)
            turn = torch.polar(torch.ones(n, r // 2, dtype=torch.float64, device="cuda"),
                               torch.outer(t.double(), s["inv_freq"].double()))[:, None]
            rows = slice(first[b], first[b] + n)

            def turned(x):
                x = x[rows].double()
                pairs = x[..., :r].unflatten(-1, (2, r // 2) if case["style"] == "halves" else (r // 2, 2))
                if case["style"] == "halves":
                    pairs = pairs.transpose(-1, -2)
                pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
                if case["style"] == "halves":
                    pairs = pairs.transpose(-1, -2)
                return torch.cat([pairs.flatten(-2), x[..., r:]], -1)
            turned_q[rows] = turned(s["q"])
            f = slots(b, t)
            p, o = torch.div(f, case["page"], rounding_mode="floor"), f % case["page"]
            for to, new, scale in ((got[0], turned(s["k"]), s["scale_k"]),
                                   (got[1], s["v"][rows].double(), s["scale_v"])):
                if scale is not None:
                    grid = _grid(case["cache"])
                    y = new / scale.double()[:, None]
                    a = y.abs().contiguous()
                    up = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)     # grid[up] >= a
                    down = (up - 1).clamp(min=0)
                    over, under = grid[up] - a, a - grid[down]
                    # a tie goes to the even code
                    pick = torch.where((over < under) | ((over == under) & (up % 2 == 0)), up, down)
                    new = torch.where(a >= grid[-1], grid[-1], grid[pick]) * torch.sign(y)
                if hnd:
                    to.transpose(1, 2)[p, o] = new
                else:
                    to[p, o] = new
        return turned_q, got[0], got[1]
    if 4.0 * D * Hq * sum(n * total for n, total in zip(q_lens, kv_lens)) > 6e12:
        return None
    T = sum(q_lens)
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    G = Hq // H

    def cached(name, b, h, start, stop):
        """Float64 (stop - start, D) of head h of tokens start .. stop - 1."""
        if case["op"] == "prompt":
            return s[name][first[b] + start: first[b] + stop, h].double()
        t = torch.arange(start, stop, device="cuda")
        f = slots(b, t)
        if case["op"] == "shared":
            n = s["shared_of"][b]
            if start < n:
                f = torch.cat([slots(s["leader"][b], t[: max(0, n - start)]), f[max(0, n - start):]])
        x = s["pages_" + name]
        x = x[:, h].reshape(-1, D) if hnd else x[:, :, h].reshape(-1, D)
        x = x.view(torch.uint8)[f].view(x.dtype) if case["cache"] != "same" else x[f]
        scale = s["scale_" + name]
        return x.double() if scale is None else x.double() * float(scale[h])

    for b, (n, total) in enumerate(zip(q_lens, kv_lens)):
        off = total - n
        for h in range(H):
            for i in range(0, n, 2048):                # rows i .. of every head of the group
                j = min(n, i + 2048)
                start, head = 0, 0
                if "window" in case:
                    start = max(0, off + i - case["window"] + 1)
                    head = min(case["sinks"], start)
                spans = ([(0, head)] if head else []) + [(start, off + j)]
                k = torch.cat([cached("k", b, h, *x) for x in spans])
                v = torch.cat([cached("v", b, h, *x) for x in spans])
                q = s["q"][first[b] + i: first[b] + j, h * G: (h + 1) * G].double()
                x = torch.einsum("igd,kd->gik", q, k) / math.sqrt(D)
                key = torch.cat([torch.arange(*x, device="cuda") for x in spans])
                row = torch.arange(off + i, off + j, device="cuda")
                gap = row[:, None] - key[None, :]
                hidden = gap < 0
                if "window" in case:
                    hidden |= (gap >= case["window"]) & (key >= case["sinks"])[None, :]
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                o = torch.einsum("gik,kd->igd", torch.exp(x - z[..., None]), v)
                out[first[b] + i: first[b] + j, h * G: (h + 1) * G] = o
                lse[first[b] + i: first[b] + j, h * G: (h + 1) * G] = z.T
    return out, lse
