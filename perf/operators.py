"""The operators of the 4-bit key/value cache, as cases to be timed and checked.

A cache holds keys and values in pages of packed 4-bit codes with one scale
(and for INT4-asym one zero-point) per group along the head dimension.  Four
operators work on it, in three kinds of case:

  append   new keys and values are coded into their pages, then read back as
           the 16-bit values they stand for
  attend   attention of new tokens' queries over the cached tokens, the
           softmax weight that each cached token drew added to its mass where
           the case asks for it
  evict    the tokens with the least mass leave the cache, the others move to
           fresh pages, which are read back

`run` has two forms: elementary torch operations in binary32 (own = False) and
the library's kernels (own = True).  `exact` is the definition in binary64.
"""

import math
import random

import torch

own = False

DEV = "cuda:0"
NF4_TABLE = (-1.0, -0.696, -0.525, -0.395, -0.284, -0.185, -0.091, 0.0,
             0.079, 0.161, 0.246, 0.338, 0.441, 0.562, 0.720, 1.0)
FP4_TABLE = tuple(s * m / 6.0 for s in (1.0, -1.0) for m in (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0))
ACT = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step of a small batch: two rows of eight heads per sequence, launch latency
        dict(name="append-token", kind="append", fmt="int4_sym", g=64, act="bf16", seqs=8, len=2048,
             new=1, heads=8, dim=128, page=64),
        # prompts of four requests entering the cache together, ragged, grouped heads
        dict(name="append-prompt", kind="append", fmt="int4_asym", g=32, act="f16", seqs=4, len=2048,
             new=2048, heads=8, dim=128, page=64),
        # one long prompt of a 7B decoder (32 heads of 128) in the library's default format
        dict(name="append-nf4", kind="append", fmt="nf4", g=64, act="bf16", seqs=1, len=8191,
             new=8191, heads=32, dim=128, page=32),
        # one chat turn at batch 1 shortly after its prompt: latency of a decode step
        dict(name="token-short", kind="attend", fmt="int4_sym", g=128, act="bf16", seqs=1, len=333,
             new=1, heads=8, group=4, dim=128, page=64, window=0, mass=False),
        # a served batch of ragged requests with grouped heads, mass kept for eviction
        dict(name="token-batch", kind="attend", fmt="int4_sym", g=64, act="bf16", seqs=32, len=4096,
             new=1, heads=8, group=4, dim=128, page=64, window=0, mass=True),
        # the same for a 7B decoder whose every head has its own keys, in the default format
        dict(name="token-7b-nf4", kind="attend", fmt="nf4", g=64, act="bf16", seqs=16, len=2048,
             new=1, heads=32, group=1, dim=128, page=32, window=0, mass=False),
        # two requests over very long documents: the length is all there is to split
        dict(name="token-long", kind="attend", fmt="int4_asym", g=32, act="f16", seqs=2, len=131071,
             new=1, heads=8, group=4, dim=128, page=128, window=0, mass=False),
        # four drafted tokens a request are verified at once, small heads, a sliding window
        dict(name="draft", kind="attend", fmt="fp4", g=32, act="f16", seqs=8, len=8192,
             new=4, heads=8, group=8, dim=64, page=16, window=4096, mass=False),
        # two whole prompts of a 7B decoder, causal: the matrix cores' case
        dict(name="prompt", kind="attend", fmt="int4_sym", g=64, act="bf16", seqs=2, len=2048,
             new=2048, heads=32, group=1, dim=128, page=64, window=0, mass=False),
        # a chunk of a long prompt after 31 chunks already cached, mass kept for eviction
        dict(name="chunk", kind="attend", fmt="int4_asym", g=64, act="bf16", seqs=1, len=32768,
             new=1024, heads=8, group=4, dim=128, page=64, window=0, mass=True),
        # one request grown past its budget by a page
        dict(name="evict-one", kind="evict", fmt="int4_sym", g=64, act="bf16", seqs=1, len=1088,
             heads=8, dim=128, page=64, budget=1024, recent=128),
        # a served batch cut to half its length
        dict(name="evict-batch", kind="evict", fmt="int4_asym", g=32, act="bf16", seqs=16, len=8192,
             heads=8, dim=128, page=64, budget=4096, recent=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "attend", "evict"])
    dim = rng.choice([64, 128, 128, 256])
    c = dict(kind=kind, fmt=rng.choice(["int4_sym", "int4_asym", "nf4", "fp4"]),
             g=rng.choice([g for g in (32, 64, 128) if g <= dim]), act=rng.choice(["f16", "bf16"]),
             seqs=_log(rng, 1, 48), heads=rng.choice([1, 2, 4, 8, 8, 32]), dim=dim,
             page=rng.choice([16, 32, 64, 128]))
    row = c["seqs"] * c["heads"] * dim  # elements per token of length
    if kind == "append":
        c["new"] = _log(rng, 1, max(1, min(8191, 2 ** 25 // row)))
        c["len"] = c["new"] + _log(rng, 1, 512)
    elif kind == "evict":
        c["len"] = _log(rng, 40, max(48, min(16384, 2 ** 27 // row)))
        c["budget"] = max(1, int(c["len"] * rng.uniform(0.3, 0.98)))
        c["recent"] = rng.randint(0, c["budget"])
    else:
        c["group"] = rng.choice([1, 2, 4, 8, 8, 16]) if c["heads"] <= 8 else 1
        c["len"] = _log(rng, 1, max(1, min(131071, 2 ** 28 // row)))
        hq = c["heads"] * c["group"]
        most = max(1, min(2048, c["len"], 2 ** 30 // (c["seqs"] * hq * max(c["len"], dim))))
        c["new"] = 1 if rng.random() < 0.4 else _log(rng, 1, most)
        c["window"] = rng.choice([0, 0, _log(rng, 16, 8192)])
        c["mass"] = rng.random() < 0.4
    return c


def _lengths(case):
    """Cached length and number of new tokens of each sequence: ragged, the first as long as the case says."""
    r = random.Random(case["len"] * 131 + case["seqs"])
    full = case.get("new") == case["len"]
    lens = [case["len"] if b == 0 else r.randint((case["len"] + 1) // 2, case["len"]) for b in range(case["seqs"])]
    most = case.get("new", 0)
    new = [n if full else (most if b == 0 else min(n, r.randint((most + 1) // 2, most))) for b, n in enumerate(lens)]
    return lens, new


# ----------------------------------------------------------- the 4-bit coding
def _levels(fmt):
    t = {"int4_sym": [i - 8.0 for i in range(16)], "int4_asym": [float(i) for i in range(16)],
         "nf4": NF4_TABLE, "fp4": FP4_TABLE}[fmt]
    return torch.tensor(t, dtype=torch.float32, device=DEV)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def _code(x, fmt, g):
    """Codes, scales and zero-points of binary32 rows x[..., D], one rounding of each quotient."""
    shape = x.shape
    x = x.reshape(*shape[:-1], shape[-1] // g, g)
    zeros = None
    if fmt == "int4_sym":
        s = (x.abs().amax(-1) / 7).clamp(max=65504.0).half()
        d = s.float()[..., None]
        c = torch.where(d > 0, torch.round(x / d).clamp(-8, 7), torch.zeros_like(x)) + 8
    elif fmt == "int4_asym":
        lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).clamp(max=65504.0).half()
        d = s.float()
        z = torch.where(d > 0, torch.round(-lo / d).clamp(0, 15), torch.zeros_like(d))
        d, zf = d[..., None], z[..., None]
        c = torch.where(d > 0, (torch.round(x / d) + zf).clamp(0, 15), torch.zeros_like(x))
        zeros = z.to(torch.uint8)
    else:
        s = x.abs().amax(-1)
        t = _levels(fmt)
        order = torch.sort(t, stable=True)
        mid = (order.values[:-1].double() + order.values[1:].double()) / 2
        q = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x))
        if fmt == "nf4":
            c = torch.bucketize(q.double(), mid)
        else:  # nearest magnitude, ties to the lower code; a magnitude of zero has code 0
            m = torch.bucketize(q.double().abs(), mid[8:])
            c = m + 8 * ((q < 0) & (m > 0))
    codes = _pack(c.reshape(shape).to(torch.uint8))
    if zeros is not None:
        zeros = torch.nn.functional.pad(zeros, (0, zeros.shape[-1] % 2))
        zeros = _pack(zeros)
    return codes, s, zeros


def _values(codes, scales, zeros, fmt, g):
    """Binary32 values [..., D] of codes [..., D/2] and their groups' scales [..., D/g]."""
    c = _unpack(codes)
    c = c.reshape(*c.shape[:-1], c.shape[-1] // g, g)
    v = _levels(fmt)[c.int()]
    if zeros is not None:
        v = v - _unpack(zeros)[..., :c.shape[-2], None].float()
    return (v * scales.float()[..., None]).flatten(-2)


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    act = ACT[case["act"]]
    H, D, page, B = case["heads"], case["dim"], case["page"], case["seqs"]
    lens, new = _lengths(case)
    per = -(-max(lens) // page)
    pages = B * per + 3
    order = torch.randperm(pages, generator=gen, device=DEV)[:B * per]
    s = dict(case)
    s["table"] = order.reshape(B, per).to(torch.int32)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def rows(n, heads, spread=1.0):
        # a few channels several times the others' size, as keys have them
        ch = 1.0 + 3.0 * (torch.rand((heads, D), generator=gen, device=DEV) < 0.04)
        return torch.randn((n, heads, D), generator=gen, device=DEV) * ch * spread

    # the cache, filled in runs of pages to bound the memory that making it takes
    s["k_codes"] = torch.empty((pages, H, page, D // 2), dtype=torch.uint8, device=DEV)
    s["v_codes"] = torch.empty_like(s["k_codes"])
    sdt = torch.float16 if case["fmt"].startswith("int4") else torch.float32
    s["k_scales"] = torch.empty((pages, H, page, D // case["g"]), dtype=sdt, device=DEV)
    s["v_scales"] = torch.empty_like(s["k_scales"])
    s["k_zeros"] = s["v_zeros"] = None
    if case["fmt"] == "int4_asym":
        s["k_zeros"] = torch.empty((pages, H, page, (D // case["g"] + 1) // 2), dtype=torch.uint8, device=DEV)
        s["v_zeros"] = torch.empty_like(s["k_zeros"])
    step = max(1, 2 ** 25 // (H * page * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        for w, spread in (("k", 1.0), ("v", 0.5)):
            x = rows(n * page, H, spread).reshape(n, page, H, D).transpose(1, 2)
            c, sc, z = _code(x, case["fmt"], case["g"])
            s[w + "_codes"][p:p + n], s[w + "_scales"][p:p + n] = c, sc
            if z is not None:
                s[w + "_zeros"][p:p + n] = z

    # which packed row is which token: sequence, place among its new tokens, position
    if case["kind"] == "evict":
        new = [min(n, case["budget"]) for n in lens]
        per2 = -(-case["budget"] // page)
        extra = pages + B * per2  # the pages that the kept tokens move to are free ones of the same pool
        for w in ("k", "v"):
            for part in ("_codes", "_scales", "_zeros"):
                t = s[w + part]
                if t is not None:
                    s[w + part] = torch.cat((t, t[:1].expand(B * per2, *t.shape[1:])))
        fresh = pages + torch.randperm(extra - pages, generator=gen, device=DEV)
        s["new_table"] = fresh.reshape(B, per2).to(torch.int32)
        s["new_lens"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        m = torch.rand((B, H, max(lens)), generator=gen, device=DEV)
        m = torch.where(m < 0.2, torch.zeros_like(m), m ** 6 * 50)  # a few heavy tokens, many that drew nothing
        s["mass"] = m
        s["width"] = case["budget"] + page
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["tokens"], s["max_new"], s["max_len"] = starts[-1], max(new), max(lens)
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
    s["seq"] = seq.to(DEV)
    s["row"] = (torch.arange(starts[-1]) - torch.tensor(starts)[seq]).to(DEV)
    s["pos"] = s["row"] + (torch.tensor(lens) - torch.tensor(new))[seq].to(DEV)
    if case["kind"] == "evict":
        s["pos"] = s["row"]
    if case["kind"] == "append":
        # slices of a fused projection's output: rows further apart than they are long
        qkv = rows(starts[-1], 2 * H + 1).to(act)
        s["k"], s["v"] = qkv[:, :H], qkv[:, H:2 * H]
    if case["kind"] == "attend":
        # queries large enough that a few keys draw most of the weight
        s["q"] = (torch.randn((starts[-1], H * case["group"], D), generator=gen, device=DEV) * 1.5).to(act)
        s["scale"] = D ** -0.5
        if case["mass"]:
            # what earlier steps left there, of the size of what one step adds
            s["mass"] = torch.rand((B, H, per * page), generator=gen, device=DEV) * (case["group"] / max(lens))
        else:
            s["mass"] = None
    return s


# --------------------------------------------------------------------- passes
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from bit_group_wise_amd import kv, q4
    if "cache" not in s:  # the handles that a serving program keeps
        s["cache"] = kv.KVCache(q4.FORMATS[s["fmt"]], s["g"], s["k_codes"], s["k_scales"], s["k_zeros"],
                                s["v_codes"], s["v_scales"], s["v_zeros"])
        if s["kind"] == "evict":
            s["batch"] = kv.Batch(s["table"], s["lens"], max_len=s["max_len"])
            s["after"] = kv.Batch(s["new_table"], s["new_lens"], s["starts"], tokens=s["tokens"],
                                  max_new=s["max_new"])
        else:
            s["batch"] = kv.Batch(s["table"], s["lens"], s["starts"] if s["max_new"] > 1 else None,
                                  tokens=s["tokens"], max_new=s["max_new"], max_len=s["max_len"])
    if s["kind"] == "append":
        kv.append(s["cache"], s["batch"], s["k"], s["v"])
        return kv.read(s["cache"], s["batch"], s["k"].dtype)
    if s["kind"] == "attend":
        out = kv.attention(s["cache"], s["batch"], s["q"], scale=s["scale"], window=s["window"], mass=s["mass"])
        return [out] if s["mass"] is None else [out, s["mass"]]
    lens, mass, kept = kv.evict(s["cache"], s["batch"], s["mass"], s["new_table"], s["budget"], s["recent"],
                                width=s["width"])
    return [lens, mass, kept, kv.read(s["cache"], s["after"], ACT[s["act"]])]


def _parts(s, w):
    return [s[w + p] for p in ("_codes", "_scales", "_zeros")]


def _slots(s, table):
    """Page and place in it of each packed row."""
    return table[s["seq"], s["pos"] // s["page"]].long(), s["pos"] % s["page"]


def _read_plain(s, table):
    page, slot = _slots(s, table)
    got = []
    for w in ("k", "v"):
        c, sc, z = (None if t is None else t[page, :, slot] for t in _parts(s, w))
        got.append(_values(c, sc, z, s["fmt"], s["g"]).to(ACT[s["act"]]))
    return tuple(got)


def _cached(s, w):
    """Values [B, H, S, D] of the pages of every sequence, S a whole number of pages."""
    t = s["table"].long()
    c, sc, z = (None if p is None else p[t].transpose(1, 2).flatten(2, 3) for p in _parts(s, w))
    return _values(c, sc, z, s["fmt"], s["g"])


def _run_plain(s):
    if s["kind"] == "append":
        page, slot = _slots(s, s["table"])
        for w in ("k", "v"):
            for to, x in zip(_parts(s, w), _code(s[w].float(), s["fmt"], s["g"])):
                if to is not None:
                    to[page, :, slot] = x
        return _read_plain(s, s["table"])
    if s["kind"] == "evict":
        return _evict_plain(s)
    B, n, H, G, D = s["seqs"], s["max_new"], s["heads"], s["group"], s["dim"]
    q = torch.zeros((B, n, H * G, D), device=DEV)
    q[s["seq"], s["row"]] = s["q"].float()
    q = q.reshape(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    k = _cached(s, "k")
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    del k
    S = x.shape[-1]
    pos = torch.full((B, n), -1, device=DEV)  # a row with no token sees nothing
    pos[s["seq"], s["row"]] = s["pos"]
    pos = pos.repeat_interleave(G, 1)[:, None, :, None]
    t = torch.arange(S, device=DEV)
    see = t <= pos
    if s["window"]:
        see &= t > pos - s["window"]
    x = torch.where(see, x, torch.full((), -math.inf, device=DEV))
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    out = torch.matmul(x, _cached(s, "v"))
    out = out.reshape(B, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, H * G, D)
    out = out[s["seq"], s["row"]].to(s["q"].dtype)
    if s["mass"] is None:
        return [out]
    s["mass"] += x.sum(2)
    return [out, s["mass"]]


def _evict_plain(s):
    B, H, L = s["mass"].shape
    n, t = s["budget"], torch.arange(L, device=DEV)
    lens = s["lens"].long()[:, None, None]
    key = torch.where(t >= lens - s["recent"], torch.full((), math.inf, device=DEV), s["mass"])
    key = torch.where(t < lens, key, torch.full((), -1.0, device=DEV))
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :n]
    m = lens.clamp(max=n)
    place = torch.arange(n, device=DEV)
    best = torch.sort(torch.where(place < m, best, torch.full((), L, device=DEV)), dim=-1).values
    live = (place < m).expand(B, H, n)
    at = torch.where(live, best, torch.zeros_like(best))
    mass = torch.where(live, torch.gather(s["mass"], 2, at), torch.zeros((), device=DEV))
    mass = torch.nn.functional.pad(mass, (0, s["width"] - n))
    kept = torch.where(live, best, torch.full((), -1, device=DEV)).int()
    b, h, _ = torch.meshgrid(torch.arange(B, device=DEV), torch.arange(H, device=DEV), place, indexing="ij")
    src = s["table"][b, at // s["page"]].long(), h, at % s["page"]
    to = s["new_table"][b, place // s["page"]].long(), h, (place % s["page"]).expand_as(at)
    src, to = [i[live] for i in src], [i[live] for i in to]
    for w in ("k", "v"):
        for part in _parts(s, w):
            if part is not None:
                part[to[0], to[1], to[2]] = part[src[0], src[1], src[2]]
    return [m[:, 0, 0].int(), mass, kept, _read_plain(s, s["new_table"])]


# ----------------------------------------------------------------------- work
def _visible(case):
    """(pairs of a new token and a cached token that it sees, cached tokens that any sees)."""
    pairs = keys = 0
    w = case["window"] or 1 << 60
    for n, m in zip(*_lengths(case)):
        first = n - m  # position of the first new token
        full = min(max(0, w - 1 - first), m)  # tokens whose window holds all before them
        pairs += sum(range(first + 1, first + full + 1)) + (m - full) * min(w, n)
        keys += n - max(0, first - w + 1)
    return pairs, keys


def work(case):
    H, D, G = case["heads"], case["dim"], case["dim"] // case["g"]
    row = D + 2 * G * (2 if case["fmt"].startswith("int4") else 4)  # bytes of a token's key and value in a head
    row += 2 * ((G + 1) // 2) if case["fmt"] == "int4_asym" else 0
    lens, new = _lengths(case)
    if case["kind"] == "append":  # the rows in, written, read, and their values out
        n = sum(new) * H
        return {"bytes": n * (4 * D + 2 * row + 4 * D), "flops": 0}
    if case["kind"] == "evict":
        kept = [min(n, case["budget"]) for n in lens]
        out = case["seqs"] * H * (case["budget"] * 4 + (case["budget"] + case["page"]) * 4)
        return {"bytes": H * (4 * sum(lens) + sum(kept) * (3 * row + 4 * D)) + out, "flops": 0}
    pairs, keys = _visible(case)
    b = keys * H * row + 4 * sum(new) * H * case["group"] * D + (8 * keys * H if case["mass"] else 0)
    return {"bytes": b, "flops": 4 * pairs * H * case["group"] * D}


# ---------------------------------------------------------------------- exact
def exact(case, seed):
    """What run() returns, from the definition in binary64, a sequence (and a head) at a time."""
    s = prepare(case, seed)
    f64 = dict(dtype=torch.float64, device=DEV)
    if case["fmt"] in ("nf4", "fp4"):  # the levels are the binary32 numbers nearest to these
        book = torch.tensor(NF4_TABLE if case["fmt"] == "nf4" else FP4_TABLE, device=DEV).double()
    else:
        book = torch.arange(16, **f64) - (8 if case["fmt"] == "int4_sym" else 0)
    g, page = case["g"], case["page"]

    def stored(w, pages, slots, h):
        """Keys or values of one head at these places, [n, D]."""
        c = s[w + "_codes"][pages, h, slots].long()
        v = torch.empty((c.shape[0], 2 * c.shape[1]), **f64)
        v[:, 0::2], v[:, 1::2] = book[c % 16], book[c // 16]
        for j in range(case["dim"] // g):
            if case["fmt"] == "int4_asym":
                z = s[w + "_zeros"][pages, h, slots, j // 2].long()
                v[:, j * g:j * g + g] -= (z // 16 if j % 2 else z % 16)[:, None]
            v[:, j * g:j * g + g] *= s[w + "_scales"][pages, h, slots, j].double()[:, None]
        return v

    def places(table, b, t):
        return table[b].long()[t // page], t % page

    lens, new = _lengths(case)
    H, B = case["heads"], case["seqs"]
    if case["kind"] == "append":
        outs = []

        def over(x, d):  # the coding rule is defined on the binary32 quotient
            return (x.float() / d.float()).double()

        for w in ("k", "v"):
            x = s[w].double()
            x = x.reshape(x.shape[0], H, -1, g)
            if case["fmt"] == "int4_sym":
                d = (x.abs().amax(-1, keepdim=True) / 7).half().double()
                y = torch.where(d > 0, torch.round(over(x, d)).clamp(-8, 7) * d, 0.0)
            elif case["fmt"] == "int4_asym":
                lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
                d = ((hi - lo) / 15).half().double()
                z = torch.round(over(-lo, d)).clamp(0, 15)
                y = torch.where(d > 0, ((torch.round(over(x, d)) + z).clamp(0, 15) - z) * d, 0.0)
            else:
                d = x.abs().amax(-1, keepdim=True)
                u = torch.where(d > 0, over(x, d), 0.0)
                best, far = torch.zeros_like(u), torch.full_like(u, math.inf)
                for level in book:
                    nearer = (u - level).abs() < far
                    best, far = torch.where(nearer, level, best), torch.where(nearer, (u - level).abs(), far)
                y = best * d
            outs.append(y.flatten(2))
        return tuple(outs)
    if case["kind"] == "evict":
        mass = torch.zeros((B, H, s["width"]), **f64)
        k, v = [], []
        host = s["mass"].cpu()
        for b, n in enumerate(lens):
            m = min(n, case["budget"])
            kb, vb = [], []
            for h in range(H):
                if n <= case["budget"]:
                    keep = list(range(n))
                else:
                    row = host[b, h, :n - case["recent"]].tolist()
                    old = sorted(range(len(row)), key=lambda t: (-row[t], t))[:m - case["recent"]]
                    keep = sorted(old) + list(range(n - case["recent"], n))
                keep = torch.tensor(keep, device=DEV)
                mass[b, h, :m] = s["mass"][b, h][keep].double()
                at = places(s["table"], b, keep)
                kb.append(stored("k", *at, h))
                vb.append(stored("v", *at, h))
            k.append(torch.stack(kb, 1))
            v.append(torch.stack(vb, 1))
        return [None, mass, None, (torch.cat(k), torch.cat(v))]
    G, first = case["group"], 0
    out = torch.zeros((s["tokens"], H * G, case["dim"]), **f64)
    mass = None if s["mass"] is None else s["mass"].double()
    for b, (n, m) in enumerate(zip(lens, new)):
        t = torch.arange(n, device=DEV)
        at = places(s["table"], b, t)
        p = torch.arange(n - m, n, device=DEV)[:, None]
        hidden = (t > p) | (t <= p - (case["window"] or n + 1))
        for h in range(H):
            kk, vv = stored("k", *at, h), stored("v", *at, h)
            for j in range(h * G, h * G + G):
                w = s["q"][first:first + m, j].double() @ kk.T * s["scale"]
                w = torch.softmax(w.masked_fill_(hidden, -math.inf), -1)
                out[first:first + m, j] = w @ vv
                if mass is not None:
                    mass[b, h, :n] += w.sum(0)
        first += m
    return [out] if mass is None else [out, mass]
