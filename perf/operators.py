"""Workloads of the paged KV cache and the dense attention over it and over packed prompts.

Four operators, named by a case's "op":

  append   new tokens' keys and values into a paged cache: quantised to 8 bits
           by their head's scale, or kept in 16
  read     tokens of a paged cache back into packed 16-bit rows
  paged    attention of each sequence's newest tokens (one, or a chunk) over
           its pages, grouped heads, bottom-right causal
  prompt   attention over packed prompts of different lengths

A case gives sizes; the sequences' lengths follow from it alone (`_lengths`),
the values from the seed.  With `own` false the operators are computed in
their plain form (elementary torch operations), with `own` true by this
repository's entry points.
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
                dim=128, page=16, layout="NHD", dtype="bf16", cache="same", causal=True)

    def case(name, op, **over):
        return {"name": name, "op": op, **base, **over}
    return [
        # one decode step of a serving batch: a token of each of 64 requests
        # goes into an 8-bit cache (latency)
        case("append_step", "append", batch=64, kv_min=500, kv_max=8192, cache="e4m3", page=64),
        # prompts of about 16k tokens in all fill an 8-bit cache
        case("append_prompts", "append", batch=12, q_min=37, q_max=4096, kv_min=37, kv_max=6000,
             cache="e4m3", page=16, layout="HND"),
        # the same into a 16-bit cache: no quantisation, pages of an odd size
        case("append_16bit", "append", batch=9, q_min=101, q_max=4001, kv_min=101, kv_max=4500,
             dtype="f16", heads=16, kv_heads=4, dim=64, page=24),
        # one request's reused prefix comes back for prompt attention
        case("read_prefix", "read", batch=1, q_min=1500, q_max=1500, kv_min=1500, kv_max=1500,
             dtype="f16", cache="e5m2", page=32),
        # whole 8-bit caches of a batch read back (a move to another layout or machine)
        case("read_caches", "read", batch=16, q_min=300, q_max=8192, kv_min=300, kv_max=8192,
             cache="e4m3", page=64, layout="HND"),
        # a few requests decoding at short context: the smallest attention call
        case("decode_few", "paged", batch=4, kv_min=100, kv_max=1024, page=16),
        # the GQA decode batch at 8k contexts of different lengths
        case("decode_batch", "paged", batch=64, kv_min=2000, kv_max=8192, page=64, layout="HND"),
        # long contexts from an 8-bit cache, eight query heads to a kv head
        case("decode_long_8bit", "paged", batch=16, kv_min=3001, kv_max=65536, heads=64,
             cache="e4m3", page=64),
        # chunked prefill: 8 requests' next tokens over their 16-bit pages
        case("chunk_16bit", "paged", batch=8, q_min=200, q_max=1024, kv_min=1024, kv_max=8192,
             page=32),
        # the same over an 8-bit cache, fewer and longer
        case("chunk_8bit", "paged", batch=3, q_min=65, q_max=2048, kv_min=2048, kv_max=16384,
             dtype="f16", cache="e4m3", page=64, layout="HND"),
        # short prompts of odd lengths, small heads
        case("prompts_short", "prompt", batch=40, q_min=1, q_max=700, lens=5, heads=12, kv_heads=4,
             dim=64, dtype="f16"),
        # one whole prompt of 16,384 tokens
        case("prompt_long", "prompt", batch=1, q_min=16384, q_max=16384, dtype="f16"),
    ]


_MOST_SCORES = 16384 * 16384 * 32     # padded scores of the largest listed case
_MOST_VALUES = 16 * 8192 * 8 * 128    # padded cache elements of the largest read / append


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("append", "read", "paged", "paged", "prompt"))
        dim = rng.choice((64, 128, 128))
        kv_heads = rng.choice((1, 2, 4, 8))
        group = rng.choice((1, 2, 3, 4, 5, 8, 16))
        c = dict(op=op, batch=_log(rng, 1, 96), q_min=1, q_max=1, kv_min=0, kv_max=0,
                 lens=rng.randrange(1, 1 << 20), heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                 page=rng.choice((16, 16, 32, 64, 64, 128, 24, 20)),
                 layout=rng.choice(("NHD", "HND")), dtype=rng.choice(("bf16", "f16")),
                 cache=rng.choice(("same", "same", "e4m3", "e5m2")), causal=rng.random() < 0.8)
        if op == "prompt":
            c["q_max"] = _log(rng, 1, 16384)
            c["q_min"] = rng.choice((c["q_max"], max(1, c["q_max"] // 9)))
        else:
            c["kv_max"] = _log(rng, 40, 65536 if op == "paged" else 8192)
            c["kv_min"] = max(1, c["kv_max"] // rng.choice((1, 4, 30)))
            if op == "read":
                c["q_max"], c["q_min"] = c["kv_max"], c["kv_min"]
            elif rng.random() < 0.6:
                c["q_max"] = min(c["kv_max"], _log(rng, 2, 4096))
                c["q_min"] = rng.choice((c["q_max"], max(1, c["q_max"] // 5)))
        keys = c["kv_max"] or c["q_max"]
        if c["batch"] * keys * kv_heads * dim > (8 * _MOST_VALUES if op == "paged" else _MOST_VALUES):
            continue
        scores = c["batch"] * c["heads"] * c["q_max"] * keys
        if op in ("paged", "prompt") and scores > _MOST_SCORES // (1 if c["causal"] else 2):
            continue
        if op in ("append", "read") and c["batch"] * keys * kv_heads * dim < 1 << 16:
            continue
        return c


def _lengths(case):
    """(new tokens, tokens in all) of each sequence."""
    r = random.Random(case["lens"])
    q = [_log(r, case["q_min"], case["q_max"]) for _ in range(case["batch"])]
    q[0] = case["q_max"]
    if case["op"] == "prompt":
        return q, list(q)
    kv = [_log(r, max(case["kv_min"], 1), case["kv_max"]) for _ in range(case["batch"])]
    kv[-1] = case["kv_max"]
    if case["op"] == "read":
        kv = list(q)
    return q, [max(a, b) for a, b in zip(q, kv)]


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

    def cumulative(lens):
        cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(lens).cumsum(0)
        return cu.cuda()
    # q, k and v of the new tokens come out of one projection
    qkv = normal(T, c["heads"] + 2 * H, D)
    s = {"case": c, "cu": cumulative(q_lens), "max_q": max(q_lens), "max_kv": max(kv_lens),
         "tokens": T, "q": qkv[:, : c["heads"]], "k": qkv[:, c["heads"]: c["heads"] + H],
         "v": qkv[:, c["heads"] + H:], "scale": 1.0 / math.sqrt(D), "scale_k": None, "scale_v": None}
    if c["op"] == "prompt":
        return s
    page, width = c["page"], -(-max(kv_lens) // c["page"])
    used = [-(-n // page) for n in kv_lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at: at + n]
        at += n
    s["table"], s["kv_lens"] = table.cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda()
    shape = (pages, page, H, D) if c["layout"] == "NHD" else (pages, H, page, D)
    s["pages_k"], s["pages_v"] = normal(*shape), normal(*shape)
    if c["cache"] != "same":
        largest = _FP8[c["cache"]][0]
        # what a calibration gives: the largest magnitude seen of each head
        amax = 3.5 + 2.5 * torch.rand(2, H, generator=g, device="cuda")
        s["scale_k"], s["scale_v"] = (amax[0] / largest).contiguous(), (amax[1] / largest).contiguous()
        for n, sc in (("pages_k", s["scale_k"]), ("pages_v", s["scale_v"])):
            by = sc.view(1, 1, H, 1) if c["layout"] == "NHD" else sc.view(1, H, 1, 1)
            s[n] = (s[n].float() / by).clamp(-largest, largest).to(_TYPES[c["cache"]])
    return s


def _places(s):
    """Page and place in it of the newest tokens of every sequence, packed."""
    cu = s["cu"].long()
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = s["kv_lens"].long()[b] - (cu[b + 1] - t)
    page = s["case"]["page"]
    return s["table"].long()[b, pos // page], pos % page


def _tokens(s, pages, scale):
    """Values of every token slot of the page table, float32 (batch, kv_heads, slots, dim)."""
    c = s["case"]
    x = pages.view(torch.uint8) if c["cache"] != "same" else pages
    x = x[s["table"].long().clamp(min=0)]                   # batch, width, page of each
    if c["cache"] != "same":
        x = x.view(_TYPES[c["cache"]])
    x = x.float()
    if c["layout"] == "NHD":
        x = x.permute(0, 3, 1, 2, 4)
    else:
        x = x.permute(0, 2, 1, 3, 4)
    x = x.reshape(c["batch"], c["kv_heads"], -1, c["dim"])
    return x if scale is None else x * scale.view(1, -1, 1, 1)


def _attend(s, k, v, kv_lens):
    """Plain attention over k, v (batch, kv_heads, keys, dim), float32, padded."""
    c = s["case"]
    B, H, D = c["batch"], c["kv_heads"], c["dim"]
    G, n = c["heads"] // H, s["max_q"]
    cu = s["cu"].long()
    q_lens = cu[1:] - cu[:-1]
    row = torch.arange(n, device="cuda")
    real = row < q_lens[:, None]                                        # batch, n
    at = (cu[:-1, None] + row).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[at].view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    x = torch.matmul(q * s["scale"], k.transpose(-1, -2)).view(B, H, G, n, -1)
    key = torch.arange(k.shape[2], device="cuda")
    seen = (key < kv_lens[:, None])[:, None, :]                         # batch, 1, keys
    if c["causal"]:
        seen = seen & (key <= (row + (kv_lens - q_lens)[:, None])[:, :, None])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m.clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H, G * n, -1), v).view(B, H, G, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, H * G, D)[real]
    return o.to(_TYPES[c["dtype"]]), lse.permute(0, 3, 1, 2).reshape(B, n, H * G)[real]


def _packed(s, x):
    """Packed rows (tokens, kv_heads, dim) as float32 (batch, kv_heads, n, dim), padded."""
    cu = s["cu"].long()
    at = (cu[:-1, None] + torch.arange(s["max_q"], device="cuda")).clamp(max=s["tokens"] - 1)
    return x.float()[at].permute(0, 2, 1, 3).contiguous()


def _put(s, pages, x, scale):
    c = s["case"]
    page, place = _places(s)
    if c["cache"] != "same":
        x = _round_fp8(x.double() / scale.double().view(1, -1, 1), c["cache"])
        x = x.float().to(_TYPES[c["cache"]]).view(torch.uint8)
    to = pages.view(torch.uint8) if c["cache"] != "same" else pages
    if c["layout"] == "NHD":
        to[page, place] = x
    else:
        to.permute(0, 2, 1, 3)[page, place] = x
    return pages


def _get(s, pages, scale):
    c = s["case"]
    page, place = _places(s)
    x = pages.view(torch.uint8) if c["cache"] != "same" else pages
    x = x[page, place] if c["layout"] == "NHD" else x.permute(0, 2, 1, 3)[page, place]
    if c["cache"] != "same":
        x = x.view(_TYPES[c["cache"]])
    x = x.float()
    return (x if scale is None else x * scale.view(1, -1, 1)).to(_TYPES[c["dtype"]])


def run(s):
    c = s["case"]
    if own:
        import sparse_attention_serving_sfa_gb300 as sfa
        if c["op"] == "prompt":
            return sfa.varlen_attention(s["q"], s["k"], s["v"], s["cu"], s["cu"], s["scale"],
                                        causal=c["causal"], return_lse=True, max_q_len=s["max_q"])
        cache = dict(kv_layout=c["layout"], scale_k=s["scale_k"], scale_v=s["scale_v"])
        if c["op"] == "append":
            sfa.paged_append(s["k"], s["v"], s["cu"], s["pages_k"], s["pages_v"], s["table"],
                             s["kv_lens"], **cache)
            return s["pages_k"], s["pages_v"]
        if c["op"] == "read":
            return sfa.paged_read(s["pages_k"], s["pages_v"], s["table"], s["kv_lens"], s["cu"],
                                  s["tokens"], dtype=c["dtype"], **cache)
        return sfa.paged_attention(s["q"], s["pages_k"], s["pages_v"], s["table"], s["kv_lens"],
                                   s["cu"], s["scale"], causal=c["causal"], return_lse=True,
                                   max_q_len=s["max_q"], **cache)
    if c["op"] == "append":
        return (_put(s, s["pages_k"], s["k"], s["scale_k"]),
                _put(s, s["pages_v"], s["v"], s["scale_v"]))
    if c["op"] == "read":
        return _get(s, s["pages_k"], s["scale_k"]), _get(s, s["pages_v"], s["scale_v"])
    if c["op"] == "paged":
        return _attend(s, _tokens(s, s["pages_k"], s["scale_k"]),
                       _tokens(s, s["pages_v"], s["scale_v"]), s["kv_lens"].long())
    cu = s["cu"].long()
    return _attend(s, _packed(s, s["k"]), _packed(s, s["v"]), cu[1:] - cu[:-1])


def work(case):
    """Each new row, and each cached token of a sequence, read or written once."""
    q_lens, kv_lens = _lengths(case)
    D, Hq, H, T = case["dim"], case["heads"], case["kv_heads"], sum(q_lens)
    cached = 2 if case["cache"] == "same" else 1
    lists = 4 * (2 * case["batch"] + 1)
    if case["op"] in ("append", "read"):
        table = 4 * sum(-(-n // case["page"]) for n in q_lens)
        return {"bytes": 2 * T * H * D * (2 + cached) + table + lists, "flops": 0}
    pairs = sum(q * kv - (q * (q - 1) // 2 if case["causal"] else 0)
                for q, kv in zip(q_lens, kv_lens))
    kv_bytes = 2 * sum(kv_lens) * H * D * (2 if case["op"] == "prompt" else cached)
    table = 0 if case["op"] == "prompt" else 4 * sum(-(-n // case["page"]) for n in kv_lens)
    return {"bytes": 2 * T * Hq * D * 2 + 4 * T * Hq + kv_bytes + table + lists,
            "flops": 4 * D * Hq * pairs}


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
    D, Hq, H, page = case["dim"], case["heads"], case["kv_heads"], case["page"]
    hnd = case["layout"] == "HND"
    first = [sum(q_lens[:b]) for b in range(len(q_lens))]

    def slots(b, start, stop):
        """Flat (page * page size + place) numbers of tokens start .. stop - 1 of sequence b."""
        t = torch.arange(start, stop, device="cuda")
        return s["table"][b].long()[torch.div(t, page, rounding_mode="floor")] * page + t % page

    def rows(pages, b, start, stop, h, scale):
        """Float64 values of head h of these tokens."""
        f = slots(b, start, stop)
        x = pages[:, h].reshape(-1, D) if hnd else pages[:, :, h].reshape(-1, D)
        x = x.view(torch.uint8)[f].view(pages.dtype) if case["cache"] != "same" else x[f]
        return x.double() if scale is None else x.double() * float(scale[h])

    if case["op"] == "append":
        got = []
        for x, pages, scale in ((s["k"], s["pages_k"], s["scale_k"]), (s["v"], s["pages_v"], s["scale_v"])):
            to = pages.double()
            for b, n in enumerate(q_lens):
                new = x[first[b]: first[b] + n].double()
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
                f = slots(b, kv_lens[b] - n, kv_lens[b])
                p, o = torch.div(f, page, rounding_mode="floor"), f % page
                if hnd:
                    to.transpose(1, 2)[p, o] = new
                else:
                    to[p, o] = new
            got.append(to)
        return tuple(got)
    if case["op"] == "read":
        return tuple(torch.cat([torch.stack([rows(pages, b, kv_lens[b] - n, kv_lens[b], h, scale)
                                             for h in range(H)], 1) for b, n in enumerate(q_lens)])
                     for pages, scale in ((s["pages_k"], s["scale_k"]), (s["pages_v"], s["scale_v"])))
    T = sum(q_lens)
    if 4.0 * D * Hq * sum(a * b for a, b in zip(q_lens, kv_lens)) > 6e12:
        return None
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    G = Hq // H
    for b, (n, total) in enumerate(zip(q_lens, kv_lens)):
        for h in range(H):
            if case["op"] == "prompt":
                k, v = (s[x][first[b]: first[b] + n, h].double() for x in "kv")
            else:
                k = rows(s["pages_k"], b, 0, total, h, s["scale_k"])
                v = rows(s["pages_v"], b, 0, total, h, s["scale_v"])
            for i in range(0, n, 2048):                # rows i .. of every head of the group
                j = min(n, i + 2048)
                last = total - n + j if case["causal"] else total
                q = s["q"][first[b] + i: first[b] + j, h * G: (h + 1) * G].double()
                x = torch.einsum("igd,kd->gik", q, k[:last]) / math.sqrt(D)
                if case["causal"]:
                    x += torch.triu(torch.full((j - i, last), -math.inf, dtype=torch.float64, device="cuda"),
                                    diagonal=total - n + i + 1)
                z = torch.logsumexp(x, -1)
                o = torch.einsum("gik,kd->igd", torch.exp(x - z[..., None]), v[:last])
                out[first[b] + i: first[b] + j, h * G: (h + 1) * G] = o
                lse[first[b] + i: first[b] + j, h * G: (h + 1) * G] = z.T
    return out, lse
