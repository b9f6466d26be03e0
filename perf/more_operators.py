"""Products through 4-bit weights whose rows fall into groups, as cases to be timed and checked.

Two things that are done beside a 4-bit weight want their rows grouped:

  experts      each row of the activations goes through the weight of its own
               expert: rows sorted by expert, groups of any size, empty ones
               among them; the rows may be gathered by an index (a token's
               copies for its experts)
  experts_dx   the gradient of that, through the frozen weights
  lora         one shared projection, and beside it each row's own low-rank
               adapter: y = x W' + s (x A') B'
  lora_bwd     its backward pass: the gradient of x through weight and
               adapter, and those of all A and B

`run` has two forms: elementary torch operations in binary32 (own = False) and
the library's kernels (own = True).  `exact` is the definition in binary64.
Every weight enters as the 16-bit value that it is dequantized to.
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
        # one decode step of eight tokens, two experts each, of a mixture with large experts
        dict(name="experts-decode", kind="experts", fmt="nf4", g=64, act="bf16", tokens=8, top=2,
             experts=8, N=14336, K=4096),
        # one token of a mixture of many small experts: most are not asked, latency counts
        dict(name="experts-token", kind="experts", fmt="int4_sym", g=128, act="f16", tokens=1, top=4,
             experts=64, N=1024, K=4096),
        # a served batch of many small experts: a few rows each
        dict(name="experts-batch", kind="experts", fmt="int4_asym", g=32, act="bf16", tokens=128, top=4,
             experts=64, N=2048, K=4096),
        # prompts through many experts: some tens to hundreds of rows each
        dict(name="experts-chunk", kind="experts", fmt="int4_sym", g=64, act="bf16", tokens=2048, top=4,
             experts=64, N=1024, K=4096),
        # prompts through large experts: the matrix cores' case
        dict(name="experts-prompt", kind="experts", fmt="int4_asym", g=32, act="bf16", tokens=2048, top=2,
             experts=8, N=14336, K=4096),
        # the gradient of a training step's prompts through frozen experts
        dict(name="experts-grad", kind="experts_dx", fmt="nf4", g=64, act="bf16", tokens=2048, top=2,
             experts=8, N=4096, K=4096),
        # a decode step of one request with its adapter
        dict(name="lora-token", kind="lora", fmt="int4_sym", g=128, act="f16", rows=1, adapters=8,
             used=1, rank=16, N=4096, K=4096),
        # a decode step of requests with an adapter each, some with none
        dict(name="lora-batch", kind="lora", fmt="nf4", g=64, act="bf16", rows=16, adapters=32,
             used=16, rank=16, N=11008, K=4096),
        # prompts of a few requests with their adapters
        dict(name="lora-prompt", kind="lora", fmt="int4_asym", g=32, act="bf16", rows=2048, adapters=8,
             used=5, rank=32, N=14336, K=4096),
        # a short fine-tuning batch of odd length
        dict(name="lora-grad-short", kind="lora_bwd", fmt="int4_sym", g=64, act="f16", rows=333, adapters=2,
             used=2, rank=8, N=1024, K=1024),
        # a fine-tuning step of one adapter on the double-quantized default
        dict(name="lora-grad", kind="lora_bwd", fmt="nf4_dq", g=64, act="bf16", rows=4096, adapters=1,
             used=1, rank=64, N=4096, K=4096),
        # the down projection of a decoder layer, two adapters trained side by side
        dict(name="lora-grad-down", kind="lora_bwd", fmt="nf4", g=64, act="bf16", rows=2048, adapters=2,
             used=2, rank=16, N=4096, K=11008),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["experts", "experts", "experts_dx", "lora", "lora", "lora_bwd"])
    g = rng.choice([32, 64, 128])
    c = dict(kind=kind, fmt=rng.choice(["nf4", "int4_sym", "int4_asym", "nf4_dq", "fp4"]), g=g,
             act=rng.choice(["f16", "bf16"]), K=g * _log(rng, max(1, 256 // g), 8192 // g))
    c["N"] = _log(rng, 64, 8192)
    if kind in ("experts_dx", "lora_bwd"):
        c["N"] = (c["N"] + 7) // 8 * 8  # rows of the gradient start at whole 16 bytes
    most = max(1, min(16384, 2 ** 37 // (c["N"] * c["K"])))  # rows that stay below the largest listed case
    if kind.startswith("experts"):
        c["experts"] = _log(rng, 1, max(1, min(128, 2 ** 28 // (c["N"] * c["K"]))))
        c["top"] = rng.randint(1, min(8, c["experts"]))
        c["tokens"] = _log(rng, 1, max(1, most // c["top"]))
    else:
        c["rows"] = _log(rng, 1, max(1, most // 2))
        c["rank"] = 8 * _log(rng, 1, 16)
        c["adapters"] = _log(rng, 1, 32 if kind == "lora" else 4)
        c["used"] = rng.randint(1, c["adapters"])
    return c


def _groups(case):
    """Rows of each expert: uneven, some popular, in small cases some empty."""
    gen = torch.Generator()
    gen.manual_seed(case["tokens"] * 131 + case["experts"])
    like = torch.exp(0.6 * torch.randn((case["experts"],), generator=gen))
    # a token's experts: `top` different ones, by exponential clocks
    clock = torch.empty((case["tokens"], case["experts"])).exponential_(generator=gen) / like
    who = torch.topk(clock, case["top"], largest=False).indices
    return torch.bincount(who.reshape(-1), minlength=case["experts"]).tolist()


def _row_ids(case):
    """The adapter of each row (-1: none): runs of a request's rows, single rows where a step decodes."""
    r = random.Random(case["rows"] * 257 + case["used"])
    who = r.sample(range(case["adapters"]), case["used"])
    if case["used"] == case["adapters"] == 1:
        return [0] * case["rows"]  # plain fine-tuning
    if case["rows"] <= 64:
        return [who[i % len(who)] if r.random() < 0.9 or i == 0 else -1 for i in range(case["rows"])]
    requests = len(who) + max(1, len(who) // 3)
    cuts = sorted(r.sample(range(1, case["rows"]), min(case["rows"] - 1, requests - 1)))
    ids = []
    for i, (lo, hi) in enumerate(zip([0] + cuts, cuts + [case["rows"]])):
        ids += [who[i] if i < len(who) else -1] * (hi - lo)
    return ids


# ----------------------------------------------------------- the 4-bit weights
def _table(fmt):
    return torch.tensor(NF4_TABLE if fmt.startswith("nf4") else FP4_TABLE, dtype=torch.float32, device=DEV)


def _pair(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _split(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def _padded(x):
    """x's flat values in storage with the padding that the library asks for (a multiple of 16 bytes, at least 16 more)."""
    size = x.element_size()
    n = ((x.numel() * size + 16 + 15) & ~15) // size
    to = torch.zeros((n,), dtype=x.dtype, device=DEV)
    to[:x.numel()] = x.reshape(-1)
    return to[:x.numel()]


def _quantized(s, case, gen, rows):
    """Codes, scales and zero-points of a random [rows, K] weight, a few outliers in it."""
    K, g, fmt = case["K"], case["g"], case["fmt"]
    s["codes"] = torch.empty((rows, K // 2), dtype=torch.uint8, device=DEV)
    sc, zp = [], []
    step = max(1, 2 ** 26 // K)
    for at in range(0, rows, step):
        n = min(step, rows - at)
        w = torch.randn((n, K // g, g), generator=gen, device=DEV) * K ** -0.5
        w.mul_(1.0 + 7.0 * (torch.rand((n, K // g, g), generator=gen, device=DEV) < 0.001)).copy_(w.half())
        if fmt == "int4_sym":
            d = (w.abs().amax(-1) / 7).half()
            c = torch.round(w / d.float()[..., None]).clamp(-8, 7) + 8
        elif fmt == "int4_asym":
            lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
            d = ((hi - lo) / 15).half()
            z = torch.round(-lo / d.float()).clamp(0, 15)
            c = (torch.round(w / d.float()[..., None]) + z[..., None]).clamp(0, 15)
            zp.append(z.to(torch.uint8).reshape(-1))
        else:
            d = w.abs().amax(-1)
            order = torch.sort(_table(fmt), stable=True)
            mid = (order.values[:-1] + order.values[1:]) / 2
            c = order.indices[torch.bucketize(w / d[..., None], mid)]
        s["codes"][at:at + n] = _pair(c.reshape(n, K).to(torch.uint8))
        sc.append(d.reshape(-1))
    sc, s["zeros"] = torch.cat(sc), None
    if fmt == "int4_asym":
        z = torch.cat(zp)
        s["zeros"] = _padded(_pair(torch.nn.functional.pad(z, (0, z.numel() % 2))))
    if fmt == "nf4_dq":  # the absmax values once more in 8 bits, a constant per run of 256
        n = sc.numel()
        runs = torch.nn.functional.pad(sc, (0, -n % 256)).reshape(-1, 256)
        s2 = runs.amax(-1) / 127
        qc = torch.round(runs / s2[:, None]).clamp(0, 127).to(torch.uint8).reshape(-1)[:n]
        s["scales"] = _padded(torch.cat((torch.nn.functional.pad(qc, (0, -n % 16)), s2.view(torch.uint8))))
    else:
        s["scales"] = _padded(sc).reshape(rows, K // g)


def _weight(s):
    """The weight [rows, K] in binary32, every value rounded to the activations' type."""
    rows, K, g, fmt = s["codes"].shape[0], s["K"], s["g"], s["fmt"]
    c = _split(s["codes"]).reshape(rows, K // g, g)
    if fmt == "int4_sym":
        w = (c.float() - 8.0) * s["scales"].float()[..., None]
    elif fmt == "int4_asym":
        z = _split(s["zeros"])[:rows * (K // g)].reshape(rows, K // g, 1).float()
        w = (c.float() - z) * s["scales"].float()[..., None]
    else:
        d = s["scales"]
        if fmt == "nf4_dq":
            n = rows * (K // g)
            s2 = d[(n + 15) // 16 * 16:].view(torch.float32)
            d = (d[:n].float() * s2.repeat_interleave(256)[:n]).reshape(rows, K // g)
        w = _table(fmt)[c.int()] * d[..., None]
    return w.to(ACT[s["act"]]).float().reshape(rows, K)


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    act, N, K = ACT[case["act"]], case["N"], case["K"]
    s = dict(case)

    def normal(*shape, size=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * size).to(act)

    if case["kind"].startswith("experts"):
        n = _groups(case)
        offsets = [0]
        for m in n:
            offsets.append(offsets[-1] + m)
        s["rows"], s["most"] = offsets[-1], max(n)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        expert = torch.repeat_interleave(torch.arange(case["experts"]), torch.tensor(n))
        s["expert"] = expert.to(DEV)
        s["place"] = (torch.arange(s["rows"]) - torch.tensor(offsets)[expert]).to(DEV)
        _quantized(s, case, gen, case["experts"] * N)
        if case["kind"] == "experts":
            s["x"] = normal(case["tokens"], K)
            # each token once for each of its experts, in an order of the seed's own
            copies = torch.arange(s["rows"], device=DEV) % case["tokens"]
            s["index"] = copies[torch.randperm(s["rows"], generator=gen, device=DEV)].to(torch.int32)
        else:
            s["dy"] = normal(s["rows"], N)
        return s
    rows, R = case["rows"], case["rank"]
    ids = _row_ids(case)
    s["ids"] = None if case["adapters"] == 1 and min(ids) == 0 else torch.tensor(ids, dtype=torch.int32, device=DEV)
    _quantized(s, case, gen, N)
    s["x"] = normal(rows, K)
    # trained adapters: their product is a fraction of the weight's
    s["a"] = normal(case["adapters"], R, K, size=K ** -0.5)
    s["b"] = normal(case["adapters"], N, R, size=0.3 * R ** -0.5)
    s["scale"] = 0.5 + 1.5 * torch.rand((case["adapters"],), generator=gen, device=DEV)
    if case["kind"] == "lora_bwd":
        s["dy"] = normal(rows, N)
    return s


# --------------------------------------------------------------------- passes
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from bit_group_wise_amd import experts, lora, q4
    if "weight" not in s:  # the handles that a user's program keeps
        s["weight"] = q4.QuantizedWeight(q4.FORMATS[s["fmt"]], s["g"], s["codes"].shape[0], s["K"], s["codes"],
                                         s["scales"], s["zeros"])
        if "a" in s:
            s["pairs"] = lora.Adapters(s["a"], s["b"], s["scale"])
    if s["kind"] == "experts":
        return experts.gemm(s["x"], s["weight"], s["offsets"], index=s["index"])
    if s["kind"] == "experts_dx":
        return experts.gemm_dx(s["dy"], s["weight"], s["offsets"])
    if s["kind"] == "lora":
        return lora.gemm(s["x"], s["weight"], s["pairs"], s["ids"])
    return lora.backward(s["dy"], s["x"], s["weight"], s["pairs"], s["ids"])


def _run_plain(s):
    w, act = _weight(s), ACT[s["act"]]
    if s["kind"].startswith("experts"):
        w = w.reshape(s["experts"], s["N"], s["K"])
        if s["kind"] == "experts":
            x, w = s["x"].float()[s["index"].long()], w.transpose(1, 2)
        else:
            x = s["dy"].float()
        full = torch.zeros((s["experts"], s["most"], x.shape[1]), device=DEV)
        full[s["expert"], s["place"]] = x
        return torch.matmul(full, w)[s["expert"], s["place"]].to(act)
    Ad, R, x = s["adapters"], s["rank"], s["x"].float()
    a = s["a"].float().reshape(Ad * R, s["K"])
    b = s["b"].float().permute(0, 2, 1).reshape(Ad * R, s["N"])
    ids = torch.zeros((s["rows"],), device=DEV) if s["ids"] is None else s["ids"]
    mine = torch.arange(Ad, device=DEV) == ids[:, None]  # no row belongs to two
    mine = (mine * s["scale"]).repeat_interleave(R, 1)
    h = (x @ a.T) * mine
    if s["kind"] == "lora":
        return (x @ w.T + h @ b).to(act)
    dy = s["dy"].float()
    u = (dy @ b.T) * mine
    dx = dy @ w + u @ a
    da = (u.T @ x).reshape(Ad, R, s["K"])
    db = (dy.T @ h).reshape(s["N"], Ad, R).permute(1, 0, 2)
    return tuple(t.to(act).contiguous() for t in (dx, da, db))


# ----------------------------------------------------------------------- work
def _weight_bytes(case, rows):
    groups = rows * (case["K"] // case["g"])
    each = {"nf4": 4.0, "fp4": 4.0, "nf4_dq": 1.0 + 4.0 / 256, "int4_sym": 2.0, "int4_asym": 2.5}[case["fmt"]]
    return int(rows * case["K"] / 2 + groups * each)


def work(case):
    N, K = case["N"], case["K"]
    if case["kind"].startswith("experts"):
        n = _groups(case)
        rows = sum(n)
        b = _weight_bytes(case, N * sum(1 for m in n if m))
        b += 2 * (min(rows, case["tokens"]) * K + rows * N) if case["kind"] == "experts" else 2 * rows * (N + K)
        return {"bytes": b, "flops": 2 * rows * N * K}
    rows, R, ids = case["rows"], case["rank"], _row_ids(case)
    low = sum(1 for i in ids if i >= 0)
    pairs = 2 * len({i for i in ids if i >= 0}) * R * (N + K)
    b = _weight_bytes(case, N) + pairs + 2 * rows * (N + K)
    if case["kind"] == "lora":
        return {"bytes": b, "flops": 2 * rows * N * K + 2 * low * R * (N + K)}
    b += 2 * case["adapters"] * R * (N + K) + 2 * rows * K  # the gradients of A and B, and x beside the gradient of x
    return {"bytes": b, "flops": 2 * rows * N * K + low * R * (4 * N + 6 * K)}


# ---------------------------------------------------------------------- exact
def exact(case, seed):
    """What run() returns, from the definition in binary64, an expert or an adapter at a time."""
    s = prepare(case, seed)
    fmt, g, K, N = case["fmt"], case["g"], case["K"], case["N"]
    groups = K // g
    levels = {"int4_sym": [i - 8 for i in range(16)], "int4_asym": list(range(16)), "fp4": FP4_TABLE}.get(fmt, NF4_TABLE)
    # the table's levels are the binary32 numbers nearest to these
    levels = torch.tensor(levels, dtype=torch.float32, device=DEV).double()

    def values(first, n):
        """Rows first .. first + n - 1 of the weight: a product in binary32, rounded to 16 bits."""
        at = torch.arange(first * groups, (first + n) * groups, device=DEV)
        if fmt == "nf4_dq":
            start = (s["codes"].shape[0] * groups + 15) // 16 * 16
            s2 = s["scales"][start:].view(torch.float32)
            d = (s["scales"][at].float() * s2[at // 256]).double()
        else:
            d = s["scales"].reshape(-1)[at].double()
        c = s["codes"][first:first + n].long()
        v = torch.empty((n, K), dtype=torch.float64, device=DEV)
        v[:, 0::2], v[:, 1::2] = levels[c % 16], levels[c // 16]
        v = v.reshape(n * groups, g)
        if fmt == "int4_asym":
            z = s["zeros"][at // 2].long()
            v -= torch.where(at % 2 == 0, z % 16, z // 16)[:, None]
        v *= d[:, None]
        return v.float().to(ACT[case["act"]]).double().reshape(n, K)

    if case["kind"].startswith("experts"):
        out, first = [], 0
        for e, n in enumerate(_groups(case)):
            if n:
                w, at = values(e * N, N), slice(first, first + n)
                out.append(s["x"][s["index"][at].long()].double() @ w.T if case["kind"] == "experts"
                           else s["dy"][at].double() @ w)
            first += n
        return torch.cat(out)
    w, x = values(0, N), s["x"].double()
    ids = torch.tensor(_row_ids(case), device=DEV)
    if case["kind"] == "lora":
        y = x @ w.T
        for i in range(case["adapters"]):
            m = (ids == i).nonzero()[:, 0]
            y[m] += s["scale"][i].double() * (x[m] @ s["a"][i].double().T) @ s["b"][i].double().T
        return y
    dy = s["dy"].double()
    dx = dy @ w
    da, db = torch.zeros_like(s["a"], dtype=torch.float64), torch.zeros_like(s["b"], dtype=torch.float64)
    for i in range(case["adapters"]):
        m = (ids == i).nonzero()[:, 0]
        u = s["scale"][i].double() * dy[m] @ s["b"][i].double()
        dx[m] += u @ s["a"][i].double()
        da[i] = u.T @ x[m]
        db[i] = dy[m].T @ (x[m] @ s["a"][i].double().T) * s["scale"][i].double()
    return dx, da, db
