"""The serving operators over compressed caches, as measured: attention for a batch that shares a
long compressed prefix (shared), decode attention that adds up each cached token's softmax weight
(weigh), and eviction of the lightest tokens into a smaller cache (evict).

``run`` computes each operator in its plain form (elementary torch operations in 32 bits) or,
where ``own`` is true, by the library's call.  A cache holds, per token and KV head, bit planes of
the key's and the value's codebook indices (32 coordinates a word group), the signs of the key's
residual projection, and 16-bit norms.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# positive halves of the Lloyd-Max centroids of N(0, 1), for 1 to 4 bits
LEVELS = {
    1: [0.7978845608028654],
    2: [0.4527800346364921, 1.510417608499096],
    3: [0.24509417894422184, 0.7560052812058781, 1.3439092785050006, 2.1519457045369874],
    4: [0.1283950298511473, 0.38804829949029174, 0.6567591185324646, 0.9423404564869629,
        1.2562311973471783, 1.6180463860218823, 2.069017226531386, 2.732589570995161],
}


def listed():
    """The measured cases: the smallest calls, ordinary ones and the largest of each operator."""
    return [
        # a single request early in its answer: latency
        dict(name="weigh one short request", op="weigh", dtype="f16", d=128, bits=3, B=1, Hq=16, Hkv=4, Nq=1,
             t_cap=200, fill=1.0),
        # a serving batch of grouped-query decode, requests of all ages
        dict(name="weigh batch of 32", op="weigh", dtype="bf16", d=128, bits=3, B=32, Hq=32, Hkv=8, Nq=1,
             t_cap=8192, fill=0.5),
        # the wide-head decode workload at 4 bits: long contexts, full caches
        dict(name="weigh wide heads, long", op="weigh", dtype="f16", d=256, bits=4, B=8, Hq=16, Hkv=4, Nq=1,
             t_cap=65536, fill=1.0),
        # two KV heads, eight query heads each, activations kept in 32 bits, an odd capacity
        dict(name="weigh in 32 bits, two heads", op="weigh", dtype="f32", d=128, bits=4, B=4, Hq=16, Hkv=2, Nq=1,
             t_cap=4099, fill=0.7),
        # four requests on a short system prompt: latency
        dict(name="shared short prompt", op="shared", dtype="f16", d=128, bits=3, B=4, Hq=16, Hkv=4, Nq=1,
             t_prefix=1000, t_cap=64, fill=0.5),
        # a serving batch on one system prompt with tools and examples
        dict(name="shared batch of 32", op="shared", dtype="bf16", d=128, bits=3, B=32, Hq=32, Hkv=8, Nq=1,
             t_prefix=8192, t_cap=512, fill=0.5),
        # many questions on one very long document
        dict(name="shared long document", op="shared", dtype="bf16", d=128, bits=3, B=64, Hq=32, Hkv=8, Nq=1,
             t_prefix=131072, t_cap=1024, fill=0.5),
        # wide heads at 2 bits on an odd prefix
        dict(name="shared wide heads", op="shared", dtype="f16", d=256, bits=2, B=16, Hq=16, Hkv=4, Nq=1,
             t_prefix=20011, t_cap=300, fill=0.6),
        # two new tokens a request (a draft to verify), narrow heads, 32-bit activations
        dict(name="shared drafts in 32 bits", op="shared", dtype="f32", d=64, bits=4, B=8, Hq=8, Hkv=2, Nq=2,
             t_prefix=3001, t_cap=100, fill=0.5),
        # one request's cache back to its budget
        dict(name="evict one short request", op="evict", d=128, bits=3, B=1, Hkv=4, t_cap=640, fill=1.0, budget=512,
             recent=64, out_cap=640),
        # a batch whose caches have grown by 256 tokens since the last eviction
        dict(name="evict batch to 4096", op="evict", d=128, bits=3, B=32, Hkv=8, t_cap=4352, fill=1.0, budget=4096,
             recent=256, out_cap=4352),
        # long prompts cut to a quarter before the answers begin
        dict(name="evict long prompts", op="evict", d=128, bits=3, B=32, Hkv=8, t_cap=32768, fill=0.8, budget=8192,
             recent=1024, out_cap=9216),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["weigh", "weigh", "shared", "shared", "evict"])
    d, bits = rng.choice([64, 128, 128, 256]), rng.choice([2, 3, 4])
    dtype = rng.choice(["f16", "bf16", "bf16", "f32"])
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 4, 7, 8])
    Nq = rng.choice([1, 1, 1, 2, 3])
    if op == "evict":
        B = _log(rng, 1, 48)
        most = 4_000_000 // (B * Hkv)
        t_cap = _log(rng, 2, min(most, 40000))
        budget = max(1, min(t_cap, int(t_cap * rng.uniform(0.1, 1.0))))
        return dict(op=op, d=d, bits=bits, B=B, Hkv=Hkv, t_cap=t_cap, fill=round(rng.uniform(0.3, 1.0), 3),
                    budget=budget, recent=int(budget * rng.uniform(0, 0.7)), out_cap=budget + rng.choice([0, 1, 40]))
    if op == "weigh":
        B = _log(rng, 1, 48)
        t_cap = _log(rng, 1, min(1_000_000 // (B * Hkv), 65536))
        return dict(op=op, dtype=dtype, d=d, bits=bits, B=B, Hq=Hkv * G, Hkv=Hkv, Nq=Nq, t_cap=t_cap,
                    fill=round(rng.uniform(0.3, 1.0), 3))
    B = _log(rng, 1, 96)
    rows = B * G * Nq * Hkv
    t_prefix = _log(rng, 16, min(100_000, 20_000_000 // rows))
    t_cap = _log(rng, 1, max(2, min(2048, 400_000 // (B * Hkv))))
    return dict(op=op, dtype=dtype, d=d, bits=bits, B=B, Hq=Hkv * G, Hkv=Hkv, Nq=Nq, t_prefix=t_prefix, t_cap=t_cap,
                fill=round(rng.uniform(0.0, 1.0), 3))


def _lens(case):
    """The tokens each sequence holds: an even spread around `fill` of the capacity (every cache is full at 1)."""
    B, cap, fill = case["B"], case["t_cap"], case["fill"]
    if fill >= 1.0:
        return [cap] * B
    w = min(fill, 1.0 - fill)
    return [min(cap, round(cap * (fill + w * (2 * ((b * 0.6180339887 + 0.5) % 1.0) - 1)))) for b in range(B)]


def _sizes(case):
    """Bytes of one token's record in a cache (one KV head), and the projection's width."""
    d, bits = case["d"], case["bits"]
    m = d // 2
    return (bits - 1) * d // 8 + m // 8 + 4 + bits * d // 8 + 2, m


def work(case):
    """Each record that the call concerns read once, each result written once; two operations for each product."""
    rec, m = _sizes(case)
    B, Hkv, d, lens = case["B"], case["Hkv"], case["d"], _lens(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        # every weight read once; a kept record and its weight read and written, its index written
        return {"bytes": Hkv * (4 * sum(lens) + kept * (2 * rec + 4 + 4)) + 8 * B, "flops": 0}
    rows = (case["Hq"] // Hkv) * case["Nq"]
    size = 4 if case["dtype"] == "f32" else 2
    io = 2 * B * Hkv * rows * d * size + 4 * B + 4 * d * (d + m)
    tokens = Hkv * sum(lens)
    if case["op"] == "weigh":
        return {"bytes": tokens * (rec + 8) + io, "flops": 2 * rows * tokens * (2 * d + m)}
    pre = case["t_prefix"] * Hkv
    return {"bytes": (tokens + pre) * rec + io, "flops": 2 * rows * (tokens + B * pre) * (2 * d + m)}


def _pack(bit):
    """[n, 32 k] truth values to [n, k] words, coordinate l of a group at bit l."""
    n, w = bit.shape
    place = torch.tensor([1 << l for l in range(32)], dtype=torch.int64, device=bit.device)
    v = (bit.view(n, w // 32, 32) * place).sum(-1)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)


def _codes(y, bits, cents):
    """Codebook indices of y [n, d] and their planar words [n, bits d / 32]."""
    idx = torch.bucketize(y, (cents[1:] + cents[:-1]) / 2)
    n, d = y.shape
    planes = torch.stack([_pack((idx >> p) & 1) for p in range(bits)], dim=-1)
    return idx, planes.reshape(n, bits * d // 32)


def prepare(case, seed):
    """Queries, weights and caches of Gaussian keys and values (as activations are after the random rotation)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = np.random.default_rng(seed)
    d, bits, B, Hkv, cap = case["d"], case["bits"], case["B"], case["Hkv"], case["t_cap"]
    m = d // 2
    qr, rr = np.linalg.qr(host.standard_normal((d, d)))
    R = torch.from_numpy((qr * np.sign(np.diag(rr))).astype(np.float32)).to(DEV)
    S = torch.from_numpy(host.standard_normal((m, d)).astype(np.float32)).to(DEV)

    def cents(b):
        c = torch.tensor(LEVELS[b], dtype=torch.float64, device=DEV) / math.sqrt(d)
        return torch.cat([-c.flip(0), c]).float()

    kc, vc = cents(bits - 1), cents(bits)
    proj = S @ R.T

    def cache(n):
        if case["op"] == "evict":  # eviction only moves the records
            word = lambda k: torch.randint(-2**31, 2**31 - 1, (n, k), generator=g, device=DEV, dtype=torch.int32)  # noqa: E731
            half = lambda: torch.rand(n, generator=g, device=DEV).half()  # noqa: E731
            return (word((bits - 1) * d // 32), word(m // 32), half(), half()), (word(bits * d // 32), half())
        got = []
        for lo in range(0, n, 1 << 19):
            k = min(n - lo, 1 << 19)
            x = torch.randn(k, d, generator=g, device=DEV)
            nk = x.norm(dim=1)
            y = x / nk[:, None]
            idx, kw = _codes(y, bits - 1, kc)
            e = y - kc[idx]
            sg = _pack((e @ proj.T >= 0).to(torch.int64))
            x = torch.randn(k, d, generator=g, device=DEV)
            nv = x.norm(dim=1)
            got.append((kw, sg, nk.half(), e.norm(dim=1).half(), _codes(x / nv[:, None], bits, vc)[1], nv.half()))
        a = [torch.cat(t).contiguous() for t in zip(*got)]
        return tuple(a[:4]), tuple(a[4:])

    s = dict(case=case, R=R, S=S, kc=kc, vc=vc, m=m)
    s["keys"], s["values"] = cache(B * Hkv * cap)
    order = host.permutation(B)
    s["lens"] = torch.tensor([_lens(case)[i] for i in order], dtype=torch.int32, device=DEV)
    if case["op"] != "shared":
        # some 16 steps' weights: a few heavy hitters and a long tail; a new token has none yet
        u = torch.randn(B, Hkv, cap, generator=g, device=DEV)
        mean = 16 * case.get("Hq", Hkv) * case.get("Nq", 1) / (Hkv * cap)
        s["weights"] = mean * torch.exp(2 * u - 2) * (torch.rand(B, Hkv, cap, generator=g, device=DEV) > 0.02)
    if case["op"] == "shared":
        s["pkeys"], s["pvalues"] = cache(Hkv * case["t_prefix"])
    if case["op"] == "evict":
        n, oc = B * Hkv, case["out_cap"]
        new = lambda t: torch.zeros((n * oc,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV)  # noqa: E731
        s["out_keys"], s["out_values"] = tuple(map(new, s["keys"])), tuple(map(new, s["values"]))
        s["out_weights"] = torch.zeros(B, Hkv, oc, device=DEV)
        s["kept"] = torch.zeros(B, Hkv, case["budget"], dtype=torch.int32, device=DEV)
        s["out_lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    else:
        s["q"] = torch.randn(B, case["Hq"], case["Nq"], d, generator=g, device=DEV).to(DTYPES[case["dtype"]])
    if own:
        from kv_cache_vector_compress_b200 import tq
        p = s["p"] = tq.Params(d, bits, m, R, S)
        if case["op"] == "weigh":
            need = tq.tq_attend_weigh_scratch_bytes(p, s["q"].dtype, B, case["Hq"], Hkv, case["Nq"], cap)
        elif case["op"] == "shared":
            need = tq.tq_attend_shared_scratch_bytes(p, s["q"].dtype, B, case["Hq"], Hkv, case["Nq"],
                                                     case["t_prefix"], cap)
        else:
            need = tq.tq_evict_scratch_bytes(p, B, Hkv, cap, case["budget"])
        s["scratch"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    return s


def _unpack(words, beta):
    """Planar words [n, beta d / 32] to codebook indices [n, d]."""
    n, w = words.shape
    bit = (words.view(n, w // beta, beta, 1) >> torch.arange(32, dtype=torch.int32, device=words.device)) & 1
    place = torch.tensor([1 << p for p in range(beta)], dtype=torch.int32, device=words.device)
    return (bit * place[:, None]).sum(2, dtype=torch.int32).view(n, 32 * w // beta)


def _scores(s, qr, qs, keys, B):
    """Estimated logits [B, Hkv, rows, T] of rotated and projected queries [B, Hkv, rows, *]."""
    Hkv = s["case"]["Hkv"]
    kw, sg, nk, rho = keys
    c = s["kc"][_unpack(kw, s["case"]["bits"] - 1).long()].view(B, Hkv, -1, qr.shape[-1])
    sign = (2 * _unpack(sg, 1) - 1).float().view(B, Hkv, -1, s["m"])
    fix = rho.float().view(B, Hkv, 1, -1) * (math.sqrt(math.pi / 2) / s["m"])
    return nk.float().view(B, Hkv, 1, -1) * (qr @ c.transpose(-1, -2) + fix * (qs @ sign.transpose(-1, -2)))


def _values(s, values, B):
    """Dequantized values in rotated coordinates, [B, Hkv, T, d]."""
    c = s["vc"][_unpack(values[0], s["case"]["bits"]).long()]
    return (values[1].float()[:, None] * c).view(B, s["case"]["Hkv"], -1, c.shape[-1])


def _plain_attend(s):
    """softmax(q k / sqrt(d)) v over the shared prefix, if there is one, and the first lens[b] cached tokens of
    each sequence; a row with nothing to attend is zero."""
    case = s["case"]
    B, Hkv, d, cap = case["B"], case["Hkv"], case["d"], case["t_cap"]
    q = s["q"].float().view(B, Hkv, -1, d)
    qr, qs = q @ s["R"].T, q @ s["S"].T
    rows = q.shape[2]
    z = _scores(s, qr, qs, s["keys"], B) / math.sqrt(d)
    there = torch.arange(cap, device=DEV) < s["lens"][:, None]
    z = torch.where(there[:, None, None], z, -math.inf)
    v = _values(s, s["values"], B)
    if case["op"] == "shared":
        fold = lambda t: t.transpose(0, 1).reshape(1, Hkv, B * rows, -1)  # noqa: E731
        unfold = lambda t: t.view(Hkv, B, rows, -1).transpose(0, 1)  # noqa: E731
        zp = unfold(_scores(s, fold(qr), fold(qs), s["pkeys"], 1) / math.sqrt(d))
        top = torch.maximum(z.amax(-1, keepdim=True), zp.amax(-1, keepdim=True))
        e, ep = torch.exp(z - top), torch.exp(zp - top)
        total = e.sum(-1, keepdim=True) + ep.sum(-1, keepdim=True)
        o = (e @ v + unfold(fold(ep) @ _values(s, s["pvalues"], 1))) / total
        return (o @ s["R"]).to(s["q"].dtype).view(s["q"].shape)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    w = e / torch.where(total == 0, 1.0, total)
    s["weights"].add_(w.sum(2))
    return [((w @ v) @ s["R"]).to(s["q"].dtype).view(s["q"].shape), s["weights"]]


def _plain_evict(s):
    """Each slice's `budget` heaviest tokens, the `recent` last ones always among them, in their order."""
    case = s["case"]
    B, Hkv, cap, budget, oc = case["B"], case["Hkv"], case["t_cap"], case["budget"], case["out_cap"]
    slot = torch.arange(cap, device=DEV)
    n = s["lens"].long()[:, None, None]
    heavy = torch.where(slot >= n - case["recent"], math.inf, s["weights"])
    heavy = torch.where(slot < n, heavy, -math.inf)
    best = torch.sort(heavy, dim=-1, descending=True, stable=True)[1][..., :budget]
    count = torch.clamp(n, max=budget)
    j = torch.arange(budget, device=DEV)
    best = torch.sort(torch.where(j < count, best, cap), dim=-1)[0]
    there = j < count
    src = (torch.arange(B * Hkv, device=DEV).view(B, Hkv, 1) * cap + best)[there.expand(B, Hkv, budget)]
    dst = (torch.arange(B * Hkv, device=DEV).view(B, Hkv, 1) * oc + j)[there.expand(B, Hkv, budget)]
    moved = list(zip(s["keys"] + s["values"] + (s["weights"].view(-1),),
                     s["out_keys"] + s["out_values"] + (s["out_weights"].view(-1),)))
    _ = [to.index_copy_(0, dst, of[src]) for of, to in moved]
    s["kept"].copy_(torch.where(there, best.int(), s["kept"]))
    s["out_lens"].copy_(count.view(B))
    return [*s["out_keys"], *s["out_values"], s["out_weights"], s["kept"], s["out_lens"]]


def run(state):
    """One pass: the plain form, or where `own` is true the library's call."""
    case = state["case"]
    if not own:
        return _plain_evict(state) if case["op"] == "evict" else _plain_attend(state)
    from kv_cache_vector_compress_b200 import tq
    s = state
    if case["op"] == "weigh":
        out = tq.tq_attend_weigh(s["p"], s["q"], s["keys"], s["values"], s["lens"], case["Hkv"], case["t_cap"],
                                 s["weights"], scratch=s["scratch"])
        return [out, s["weights"]]
    if case["op"] == "shared":
        return tq.tq_attend_shared(s["p"], s["q"], s["pkeys"], s["pvalues"], s["keys"], s["values"], s["lens"],
                                   case["Hkv"], case["t_prefix"], case["t_cap"], scratch=s["scratch"])
    tq.tq_evict(s["p"], s["keys"], s["values"], s["weights"], s["lens"], case["Hkv"], case["t_cap"], case["budget"],
                case["recent"], case["out_cap"], out_keys=s["out_keys"], out_values=s["out_values"],
                out_weights=s["out_weights"], kept=s["kept"], out_lens=s["out_lens"], scratch=s["scratch"])
    return [*s["out_keys"], *s["out_values"], s["out_weights"], s["kept"], s["out_lens"]]


def exact(case, seed):
    """The attention operators in 64 bits, from vectors put back into the original coordinates, one KV head at a
    time; eviction computes no numbers."""
    if case["op"] == "evict":
        return None
    s = prepare(case, seed)
    B, Hkv, d, bits, cap, m = case["B"], case["Hkv"], case["d"], case["bits"], case["t_cap"], s["m"]
    R, S = s["R"].double(), s["S"].double()
    shift = torch.arange(32, device=DEV)

    def table(words, beta, cents):
        w = words.view(len(words), words.shape[1] // beta, beta)
        idx = sum(((w[:, :, p, None].long() >> shift) & 1) << p for p in range(beta))
        return cents.double()[idx.view(len(words), 32 * w.shape[1])]

    def vectors(keys, values, lo, n):
        kw, sg, nk, rho = (t[lo:lo + n] for t in keys)
        vw, nv = (t[lo:lo + n] for t in values)
        sign = table(sg, 1, torch.tensor([-1.0, 1.0], device=DEV))
        unit = table(kw, bits - 1, s["kc"]) @ R + math.sqrt(math.pi / 2) / m * rho.double()[:, None] * (sign @ S)
        return nk.double()[:, None] * unit, nv.double()[:, None] * (table(vw, bits, s["vc"]) @ R)

    G = case["Hq"] // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if case["op"] == "weigh" else None
    lens = s["lens"].tolist()
    for h in range(Hkv):
        if case["op"] == "shared":
            pk, pv = vectors(s["pkeys"], s["pvalues"], h * case["t_prefix"], case["t_prefix"])
        for b in range(B):
            k, v = vectors(s["keys"], s["values"], (b * Hkv + h) * cap, lens[b])
            if case["op"] == "shared":
                k, v = torch.cat([pk, k]), torch.cat([pv, v])
            if len(k) == 0:
                continue
            q = s["q"][b, h * G:(h + 1) * G].double()
            w = torch.softmax(q @ k.T / math.sqrt(d), dim=-1)
            out[b, h * G:(h + 1) * G] = w @ v
            if weights is not None:
                weights[b, h, :lens[b]] += w.sum((0, 1))
    return out if weights is None else [out, weights]
