"""The operators of an 8-bit paged key-value cache, as cases to measure.

append   attn_sink_cache_append_fp8: new key and value rows (bf16, packed
         sequences) are quantised to e4m3 as they enter the page pools, with
         one power-of-two scale for each position and kv head.
read     attn_sink_cache_read_fp8: the last rows of every sequence come back
         out of the pools as packed bf16.
decode   attn_sink_decode_paged_fp8: one new token for each sequence attends
         to the pools (sliding window, learned sink).
extend   attn_sink_fwd_extend: packed prompt chunks attend to what came before
         them and to themselves (more keys than queries).

A row x of D channels is held as codes c (e4m3) and a scale 2^e (e8m0), e the
smallest integer in [-117, 119] with max|x| <= 448 * 2^e; c = x / 2^e rounded to
nearest even.

`own` false: the plain form, in elementary torch operations; true: the
framework's entry points on the same state.
"""
import math
import random

import torch

own = False

DEV = "cuda"
FULL = 1 << 30                        # a window that covers every sequence


# ------------------------------------------------------------------ the cases
def _case(op, B, new, past, Hkv, D, P=64, G=8, W=FULL, name=None):
    c = dict(op=op, B=B, new_lo=new[0], new_hi=new[1], past_lo=past[0], past_hi=past[1],
             Hkv=Hkv, G=G, D=D, P=P, W=W)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # every sequence of a serving batch writes the token it has just made
        _case("append", 64, (1, 1), (4096, 16384), 4, 128, 64, name="append one token"),
        # prompts of a mixed batch enter a cache of small pages
        _case("append", 24, (1, 4096), (0, 0), 4, 128, 16, name="append ragged prompts"),
        # long prompts, many kv heads, large pages: the widest write
        _case("append", 8, (15000, 16384), (0, 777), 8, 128, 256, name="append long prompts"),
        # the window's W - 1 keys before a chunk, read back for a few sequences
        _case("read", 4, (512, 512), (100, 3000), 4, 128, 64, name="read a window"),
        # prefixes of very different lengths, narrow heads
        _case("read", 24, (1, 4096), (0, 0), 2, 64, 16, name="read ragged prefixes"),
        # long prefixes of a full causal model
        _case("read", 8, (15000, 16384), (0, 777), 8, 128, 256, name="read long prefixes"),
        # a single user inside the sliding window: latency alone
        _case("decode", 1, (1, 1), (300, 2000), 4, 128, 64, W=513, name="decode one windowed"),
        # a small batch of long contexts
        _case("decode", 8, (1, 1), (4096, 131072), 4, 128, 64, name="decode 8 long"),
        # the full serving batch
        _case("decode", 64, (1, 1), (4096, 131072), 4, 128, 256, name="decode 64 long"),
        # wide heads, small pages, an odd group
        _case("decode", 32, (1, 1), (1, 32768), 2, 256, 16, G=5, name="decode wide heads"),
        # the next chunks of windowed prompts: 512 earlier keys for each chunk
        _case("extend", 4, (700, 1024), (512, 512), 4, 128, W=513, name="extend windowed chunks"),
        # a chunk late in a long prompt, full causal
        _case("extend", 1, (4096, 4096), (12288, 12288), 8, 128, G=4, name="extend a long prompt"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _plain_elements(c):
    """Elements of the largest intermediate of the plain form."""
    n_hi = c["past_hi"] + (0 if c["op"] == "decode" else c["new_hi"])
    if c["op"] == "decode":
        return c["B"] * min(c["W"], n_hi + c["P"]) * c["Hkv"] * c["D"]
    if c["op"] == "extend":
        return c["B"] * c["Hkv"] * c["G"] * c["new_hi"] * n_hi
    return c["B"] * c["new_hi"] * c["Hkv"] * c["D"]


def _too_large(c):
    """Whether a drawn case costs more than the largest listed one of its operator."""
    top = [x for x in listed() if x["op"] == c["op"]]
    cost = lambda x: max(work(x)["bytes"], work(x)["flops"] / 200)  # noqa: E731
    return cost(c) > max(map(cost, top)) or _plain_elements(c) > max(map(_plain_elements, top)) or \
        c["B"] * (c["past_hi"] + c["new_hi"] + c["P"]) * c["Hkv"] * c["D"] > 64 * 131072 * 512


def draw(rng):
    op = rng.choice(["append", "read", "decode", "extend"])
    D = rng.choice([64, 128, 256])
    G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8] if D == 256 else [1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    Hkv = _log_int(rng, 1, 8)
    P = 1 << rng.randint(4, 9)
    W = rng.choice([_log_int(rng, 1, 8192), 513, FULL, FULL])
    B = _log_int(rng, 1, 256)
    if op == "decode":
        new = (1, 1)
        hi = _log_int(rng, 1, 131072)
        past = (rng.choice([1, max(1, hi // 4), hi]), hi)
    elif op == "extend":
        hi = _log_int(rng, 1, 4096)
        new = (rng.choice([1, max(1, hi // 2), hi]), hi)
        hi = _log_int(rng, 1, 12288)
        past = (rng.choice([0, hi // 2, hi]), hi)
        B = _log_int(rng, 1, 24)
    else:
        hi = _log_int(rng, 1, 16384)
        new = (rng.choice([1, max(1, hi // 2), hi]), hi)
        hi = _log_int(rng, 1, 8192)
        past = (rng.choice([0, hi // 2, hi]), hi)
    c = _case(op, B, new, past, Hkv, D, P, G, W)
    while _too_large(c):
        if c["B"] > 1:
            c["B"] = c["B"] * 2 // 3
        else:
            for k in ("new_lo", "new_hi", "past_lo", "past_hi"):
                c[k] = c[k] * 2 // 3 if c[k] > 1 else c[k]
    return c


def _lengths(c):
    """(new rows, earlier rows) of every sequence; they belong to the case, not to the seed."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    past = [r.randint(c["past_lo"], c["past_hi"]) for _ in range(c["B"])]
    return new, past


def work(c):
    new, past = _lengths(c)
    Hkv, D, Hq, W, P = c["Hkv"], c["D"], c["Hkv"] * c["G"], c["W"], c["P"]
    if c["op"] in ("append", "read"):
        # bf16 rows on one side, codes and a scale byte on the other; K and V
        rows = sum(new)
        pages = sum((past[b] + new[b] - 1) // P - past[b] // P + 1 for b in range(c["B"]))
        return {"bytes": 2 * rows * Hkv * (2 * D + D + 1) + 4 * pages + 8 * c["B"], "flops": 0}
    if c["op"] == "decode":
        seen = [min(n, W) for n in past]
        pages = sum((n - 1) // P - (n - s) // P + 1 for n, s in zip(past, seen))
        return {"bytes": 2 * sum(seen) * Hkv * (D + 1) + 4 * c["B"] * Hq * D + 4 * pages + 4 * c["B"] + 4 * Hq,
                "flops": 4 * D * Hq * sum(seen)}
    pairs = 0
    for n, p in zip(new, past):
        full = min(n, max(0, p + n - W + 1)) if W > p else n            # queries that see W keys
        short = n - full                                                 # they see p + 1 .. p + short
        pairs += full * W + short * p + short * (short + 1) // 2
    T, Tk = sum(new), sum(n + min(p, W - 1) for n, p in zip(new, past))
    return {"bytes": 2 * 2 * T * Hq * D + 2 * 2 * Tk * Hkv * D + 4 * T * Hq + 8 * c["B"] + 4 * Hq,
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ the state
def _pools(c, total, g):
    """Page pools holding quantised rows in every position, and the table of every sequence's pages
    (in no order) for `total` positions each.  Entries past a sequence's last page are -1."""
    B, Hkv, D, P = c["B"], c["Hkv"], c["D"], c["P"]
    pages = [-(-n // P) for n in total]
    MP, NB = max(1, max(pages)), sum(pages) + 3
    table = torch.full((B, MP), -1, dtype=torch.int32)
    order = torch.randperm(NB, generator=torch.Generator().manual_seed(int(g.initial_seed()) + 1)).to(torch.int32)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = order[at: at + m]
        at += m
    pools = []
    per = max(1, (1 << 26) // (P * Hkv * D))
    for kind in range(2):
        codes = torch.empty(NB, P, Hkv, D, dtype=torch.uint8, device=DEV)
        scales = torch.empty(NB, Hkv, P, dtype=torch.uint8, device=DEV)
        head = torch.randn(Hkv, 1, generator=g, device=DEV).mul_(0.5).exp2_()
        for i in range(0, NB, per):
            x = torch.randn(min(per, NB - i), P, Hkv, D, generator=g, device=DEV) * head
            if kind:                                     # value rows of different sizes
                x *= torch.randn(x.shape[0], P, Hkv, 1, generator=g, device=DEV).mul_(0.7).exp2_()
            codes[i: i + per], s = _quantise(x)
            scales[i: i + per] = s.transpose(1, 2)
        pools += [codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)]
    return pools[0], pools[2], pools[1], pools[3], table.to(DEV)


def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    new, past = _lengths(c)
    op, B, Hkv, D, W = c["op"], c["B"], c["Hkv"], c["D"], c["W"]
    Hq = Hkv * c["G"]
    bf = torch.bfloat16
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = {"op": op, "W": W, "scale": 1.0 / math.sqrt(D)}
    if op in ("append", "read"):
        total = [p + n for p, n in zip(past, new)]
        s["kp"], s["vp"], s["ks"], s["vs"], s["table"] = _pools(c, total, g)
        s["seqlens"] = torch.tensor(total, dtype=torch.int32, device=DEV)
        s["cu"] = _cu(new)
        T = sum(new)
        if op == "append":
            s["k"] = (randn(T, Hkv, D) * randn(Hkv, 1).mul_(0.5).exp2_()).to(bf)
            s["v"] = (randn(T, Hkv, D) * randn(T, Hkv, 1).mul_(0.7).exp2_()).to(bf)
        else:
            s["k"] = torch.empty(T, Hkv, D, dtype=bf, device=DEV)
            s["v"] = torch.empty(T, Hkv, D, dtype=bf, device=DEV)
        return s
    s["sinks"] = torch.rand(Hq, generator=g, device=DEV) * 12 - 4
    if op == "decode":
        s["kp"], s["vp"], s["ks"], s["vs"], s["table"] = _pools(c, past, g)
        s["seqlens"] = torch.tensor(past, dtype=torch.int32, device=DEV)
        s["q"] = (randn(B, Hq, D) * 1.5).to(bf)
        s["out"] = torch.empty(B, Hq, D, dtype=bf, device=DEV)
        return s
    T, Tk = sum(new), sum(new) + sum(past)
    s["cu_q"], s["cu_k"], s["Lq"] = _cu(new), _cu([p + n for p, n in zip(past, new)]), max(new)
    s["Lk"] = max(p + n for p, n in zip(past, new))
    s["q"], s["k"], s["v"] = (randn(T, Hq, D) * 1.5).to(bf), randn(Tk, Hkv, D).to(bf), randn(Tk, Hkv, D).to(bf)
    s["out"] = torch.empty(T, Hq, D, dtype=bf, device=DEV)
    s["lse"] = torch.empty(Hq, T, dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------- the plain form
def _quantise(x):
    """Codes (e4m3 bytes) and scale bytes (e8m0) of the rows of x (f32)."""
    top = x.abs().amax(-1)
    mant, ex = torch.frexp(top)
    e = torch.where(top > 0, ex - 9 + (mant > 0.875), -117).clamp(-117, 119)   # 448 = 0.875 * 2^9
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _places(s):
    """(page, position in page) of every packed row: the last rows of its sequence."""
    cu, P = s["cu"].long(), s["kp"].shape[1]
    T = s["k"].shape[0]
    r = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu, r, right=True) - 1
    pos = s["seqlens"].long()[b] - (cu[b + 1] - r)
    return s["table"].long()[b, pos // P], pos % P


def _values(codes, scales):
    return codes.to(torch.float32) * scales.to(torch.float32)[..., None]


def _plain_append(s):
    page, at = _places(s)
    for x, pool, scales in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        codes, e = _quantise(x.float())
        pool.view(torch.uint8)[page, at] = codes
        scales.view(torch.uint8)[page, :, at] = e
    return s["kp"], s["vp"], s["ks"], s["vs"]


def _plain_read(s):
    page, at = _places(s)
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    u8 = lambda t: t.view(torch.uint8)  # noqa: E731
    k = _values(u8(s["kp"])[page, at].view(e4), u8(s["ks"])[page, :, at].view(e8))
    v = _values(u8(s["vp"])[page, at].view(e4), u8(s["vs"])[page, :, at].view(e8))
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_decode(s):
    q, sinks = s["q"].float(), s["sinks"]
    B, Hq, D = q.shape
    P, Hkv, MP = s["kp"].shape[1], s["kp"].shape[2], s["table"].shape[1]
    span = min(s["W"], MP * P)
    n = s["seqlens"].long()
    pos = n[:, None] - span + torch.arange(span, device=DEV)            # the last `span` positions
    seen = pos >= 0
    pos = pos.clamp(min=0)
    page, at = s["table"].long().gather(1, pos // P), pos % P
    page = page.clamp(min=0)
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu

    def rows(pool, scales):                                             # [B, Hkv, span, D]
        x = _values(pool.view(torch.uint8)[page, at].view(e4), scales.view(torch.uint8)[page, :, at].view(e8))
        return x.transpose(1, 2)

    qg = q.view(B, Hkv, Hq // Hkv, D)
    sc = torch.matmul(qg, rows(s["kp"], s["ks"]).transpose(-1, -2)) * s["scale"]
    sc = sc.masked_fill(~seen[:, None, None, :], -math.inf)
    sink = sinks.view(1, Hkv, -1, 1)
    m = torch.maximum(sc.amax(-1, keepdim=True), sink)
    p = torch.exp(sc - m)
    den = p.sum(-1, keepdim=True) + torch.exp(sink - m)
    o = torch.matmul(p, rows(s["vp"], s["vs"])) / den
    return o.view(B, Hq, D).to(torch.bfloat16)


def _plain_extend(s):
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    T, Hq, D = s["q"].shape
    Hkv = s["k"].shape[1]
    B, Lq, Lk = cq.shape[0] - 1, s["Lq"], s["Lk"]
    nq, nk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    i, j = torch.arange(Lq, device=DEV), torch.arange(Lk, device=DEV)
    qi = (cq[:-1, None] + i).clamp(max=T - 1)
    kj = (ck[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    q = s["q"].float()[qi].view(B, Lq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[kj].permute(0, 2, 3, 1)[:, :, None]              # [B, Hkv, 1, D, Lk]
    v = s["v"].float()[kj].permute(0, 2, 1, 3)[:, :, None]
    sc = torch.matmul(q, k).mul_(s["scale"])                            # [B, Hkv, G, Lq, Lk]
    at = (i + (nk - nq)[:, None])[:, :, None]                           # each query's position
    hidden = (j > at) | (j <= at - s["W"]) | (i >= nq[:, None])[:, :, None]
    sc = sc.masked_fill_(hidden[:, None, None], -math.inf)
    sink = s["sinks"].view(1, Hkv, -1, 1, 1)
    m = torch.maximum(sc.amax(-1, keepdim=True), sink)
    p = sc.sub_(m).exp_()
    den = p.sum(-1, keepdim=True) + torch.exp(sink - m)
    o = torch.matmul(p, v) / den
    lse = (m + torch.log(den)).view(B, Hq, Lq)
    r = torch.arange(T, device=DEV)
    b = torch.searchsorted(cq, r, right=True) - 1
    o = o.reshape(B, Hq, Lq, D)[b, :, r - cq[b]]
    return o.to(torch.bfloat16), lse[b, :, r - cq[b]].t().contiguous()


def run(s):
    op = s["op"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "decode": _plain_decode, "extend": _plain_extend}[op](s)
    import sliding_window_learned_b200 as swl
    if op == "append":
        swl.attn_sink_cache_append_fp8(s["k"], s["v"], s["table"], s["seqlens"], s["cu"],
                                       s["kp"], s["vp"], s["ks"], s["vs"])
        return s["kp"], s["vp"], s["ks"], s["vs"]
    if op == "read":
        swl.attn_sink_cache_read_fp8(s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["seqlens"], s["cu"],
                                     s["k"], s["v"])
        return s["k"], s["v"]
    if op == "decode":
        swl.attn_sink_decode_paged_fp8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["seqlens"],
                                       s["sinks"], s["W"], s["scale"], s["out"])
        return s["out"]
    swl.attn_sink_fwd_extend(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["Lq"], s["sinks"], s["W"],
                             s["scale"], s["out"], s["lse"])
    return s["out"], s["lse"]


# ------------------------------------------------------ the definition, 64 bits
def _exact_rows(x):
    """Rows of x (f64) as held: (codes' values, scales)."""
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(top / 448)).clamp(-117, 119)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)                # log2's last bit
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e).clamp(-117, 119)
    y = x / torch.exp2(e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)   # the grid at y
    return torch.round(y / step) * step, torch.exp2(e)                  # (round: half to even)


def _sequence(s, b, n):
    """Flat positions 0 .. n-1 of sequence b as (page, position in page)."""
    P = s["kp"].shape[1]
    pos = torch.arange(n, device=DEV)
    return s["table"][b].long()[pos // P], pos % P


def exact(c, seed):
    s = prepare(c, seed)
    new, past = _lengths(c)
    op, D, W, G = c["op"], c["D"], c["W"], c["G"]
    f64 = torch.float64
    if op == "append":
        outs = [s["kp"].to(f64), s["vp"].to(f64), s["ks"].to(f64), s["vs"].to(f64)]
        row = 0
        for b, (n, p) in enumerate(zip(new, past)):
            page, at = (x[p:] for x in _sequence(s, b, p + n))
            for x, pool, scales in ((s["k"], outs[0], outs[2]), (s["v"], outs[1], outs[3])):
                pool[page, at], sc = _exact_rows(x[row: row + n].to(f64))
                scales[page, :, at] = sc
            row += n
        return tuple(outs)
    if op == "read":
        outs = [torch.empty(s["k"].shape, dtype=f64, device=DEV) for _ in range(2)]
        row = 0
        for b, (n, p) in enumerate(zip(new, past)):
            page, at = (x[p:] for x in _sequence(s, b, p + n))
            for x, pool, scales in ((outs[0], s["kp"], s["ks"]), (outs[1], s["vp"], s["vs"])):
                for h in range(c["Hkv"]):
                    x[row: row + n, h] = pool[page, at, h].to(f64) * scales[page, h, at].to(f64)[:, None]
            row += n
        return tuple(outs)
    sink = s["sinks"].to(f64)
    if op == "decode":
        out = torch.zeros(s["q"].shape, dtype=f64, device=DEV)
        for b, n in enumerate(past):
            page, at = (x[max(0, n - W):] for x in _sequence(s, b, n))
            for h in range(c["Hkv"]):
                k = s["kp"].view(torch.uint8)[page, at, h].view(torch.float8_e4m3fn).to(f64)
                k = k * s["ks"].view(torch.uint8)[page, h, at].view(torch.float8_e8m0fnu).to(f64)[:, None]
                v = s["vp"].view(torch.uint8)[page, at, h].view(torch.float8_e4m3fn).to(f64)
                v = v * s["vs"].view(torch.uint8)[page, h, at].view(torch.float8_e8m0fnu).to(f64)[:, None]
                x = s["q"][b, h * G: h * G + G].to(f64) @ k.T * s["scale"]
                x = torch.cat([x, sink[h * G: h * G + G, None]], 1)
                out[b, h * G: h * G + G] = torch.softmax(x, 1)[:, :-1] @ v
        return out
    out = torch.zeros(s["q"].shape, dtype=f64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=f64, device=DEV)
    q0 = k0 = 0
    for n, p in zip(new, past):
        at = torch.arange(p, p + n, device=DEV)[:, None]
        j = torch.arange(p + n, device=DEV)[None]
        seen = (j <= at) & (j > at - W)
        for h in range(c["Hkv"] * G):
            k = s["k"][k0: k0 + p + n, h // G].to(f64)
            x = s["q"][q0: q0 + n, h].to(f64) @ k.T * s["scale"]
            x = torch.where(seen, x, -math.inf)
            x = torch.cat([x, sink[h].expand(n, 1)], 1)
            out[q0: q0 + n, h] = torch.softmax(x, 1)[:, :-1] @ s["v"][k0: k0 + p + n, h // G].to(f64)
            lse[h, q0: q0 + n] = torch.logsumexp(x, 1)
        q0, k0 = q0 + n, k0 + p + n
    return out, lse
