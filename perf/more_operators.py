"""Cases of the operators around a decoder layer's quantized projections.

Four operators: the root-mean-square norm in front of a projection with the
residual's addition, in 16 or 32 bits or as the int8 rows that the projection
takes (``norm``); rotary positions (``rope``); queries and keys rotated on their
way into the paged cache, with the values (``place``); and low-rank adapters of
many requests beside one shared projection (``lora``).

Lengths and adapters are a fixed multiset per case (so that ``work`` knows
them), dealt in an order that the seed decides; pages lie in the pool in an
order that the seed decides too.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "int8": torch.int8}
SIZE = {"bf16": 2, "fp32": 4, "int8": 1}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's token in front of a small model's up-projection: launch latency
        dict(name="norm_token", op="norm", M=1, K=1152, x="fp32", out="int8", res=False, offset=1.0, eps=1e-6),
        # a serving step on a 7B-class layer: the residual's addition, the norm and the int8 rows of the next projection
        dict(name="norm_step", op="norm", M=64, K=4096, x="fp32", out="int8", res=True, offset=0.0, eps=1e-5),
        # prompts of a 70B-class layer in front of a weight-only projection, which takes bf16
        dict(name="norm_prompt", op="norm", M=8192, K=8192, x="fp32", out="bf16", res=True, offset=0.0, eps=1e-5),
        # one token's query and key of a small model, one joint row
        dict(name="rope_token", op="rope", T=1, heads=5, row=6, d=256, rot=256, layout="half", x="bf16", scaling="none", factor=1.0,
             far=700),
        # prompts behind a long context, neighbouring pairs in half of the head, frequencies stretched for it
        dict(name="rope_prompt", op="rope", T=8191, heads=40, row=48, d=128, rot=64, layout="pairs", x="fp32", scaling="yarn",
             factor=16.0, far=131072),
        # a serving step of ragged sequences on 7B-class layers, 8-bit cache, fp32 activations of the quantized projection
        dict(name="place_step", op="place", B=64, hq=32, hkv=8, d=128, rot=128, ps=64, max_len=8191, min_len=1, max_n=1, min_n=1,
             layout="half", scaling="none", factor=1.0, x="fp32", kv="int8"),
        # prompts written whole, heads of 80 of which 32 rotate
        dict(name="place_prompt", op="place", B=5, hq=12, hkv=4, d=80, rot=32, ps=16, max_len=9000, min_len=8, max_n=8191, min_n=7,
             layout="half", scaling="linear", factor=4.0, x="bf16", kv="bf16"),
        # chunks behind long conversations on 70B-class layers
        dict(name="place_long", op="place", B=4, hq=64, hkv=8, d=128, rot=128, ps=64, max_len=131072, min_len=60000, max_n=2048,
             min_n=1024, layout="half", scaling="bands", factor=8.0, x="fp32", kv="bf16"),
        # one user's token and one small adapter on a small model's up-projection
        dict(name="lora_token", op="lora", M=1, K=1152, N=6912, rank=8, adapters=4, none=0, x="fp32", rows="step", ragged=False),
        # a serving step of many users with adapters of their own, some without, on a 7B-class layer
        dict(name="lora_step", op="lora", M=64, K=4096, N=11008, rank=16, adapters=32, none=7, x="fp32", rows="step", ragged=True),
        # few users with large adapters beside a 70B-class weight-only layer
        dict(name="lora_wide", op="lora", M=16, K=8192, N=28672, rank=64, adapters=16, none=0, x="bf16", rows="step", ragged=False),
        # prompts of a few users on a 7B-class layer
        dict(name="lora_prompt", op="lora", M=8192, K=4096, N=4096, rank=32, adapters=5, none=0, x="fp32", rows="prompt",
             ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _stretch(rng):
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn", "bands"])
    return dict(scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 40.0]))


def draw(rng):
    op = rng.choice(["norm", "norm", "rope", "place", "place", "lora", "lora", "lora"])
    if op == "norm":
        K = rng.choice([_log(rng, 64, 16384), 8 * _log(rng, 8, 2048), 128 * _log(rng, 2, 128)])
        return dict(op=op, M=_log(rng, 1, max(2, (3 << 24) // K)), K=K, x=rng.choice(["bf16", "fp32"]),
                    out=rng.choice(["int8", "int8", "bf16", "fp32"]), res=rng.choice([True, False]), offset=rng.choice([0.0, 1.0]),
                    eps=rng.choice([1e-6, 1e-5]))
    layout = rng.choice(["half", "pairs"])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 128, 256, 72, 40])
        row = rng.choice([1, 3, 6, 12, 28, 48, 80])
        return dict(op=op, T=_log(rng, 1, min(32768, (1 << 26) // (row * d))), heads=rng.randint(1, row), row=row, d=d,
                    rot=rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]), layout=layout, x=rng.choice(["bf16", "fp32"]),
                    far=_log(rng, 100, 1000000), **_stretch(rng))
    if op == "place":
        d = rng.choice([64, 128, 128, 256, 96, 80])
        hkv = rng.choice([1, 2, 4, 8, 5])
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        B = _log(rng, 1, 128)
        new = rng.choice([1, _log(rng, 2, max(3, (1 << 25) // (B * (hq + 2 * hkv) * d)))])
        n = new + _log(rng, 1, min(100000, 400000 // B))
        return dict(op=op, B=B, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]),
                    ps=rng.choice([16, 32, 64, 128]), max_len=n, min_len=1, max_n=new, min_n=rng.choice([1, new]), layout=layout,
                    x=rng.choice(["bf16", "fp32"]), kv=rng.choice(["bf16", "int8"]), **_stretch(rng))
    rank = rng.choice([4, 8, 16, 16, 32, 64, 128, rng.randint(1, 100)])
    K, N = (rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), 128 * _log(rng, 2, 64)]) for _ in range(2))
    rows = rng.choice(["step", "step", "prompt"])
    M = _log(rng, 1, 256) if rows == "step" else _log(rng, 100, max(101, min(8192, (1 << 26) // (K + 2 * N))))
    adapters = _log(rng, 1, 64 if rows == "step" else 8)
    return dict(op=op, M=M, K=K, N=N, rank=rank, adapters=adapters, none=rng.choice([0, M // 5]), x=rng.choice(["bf16", "fp32"]),
                rows=rows, ragged=rng.choice([True, False]))


def _spread(count, lo, hi, key):
    """`count` whole numbers from lo to hi, the ends among them, the same for every seed."""
    r = random.Random("%d %d %d %s" % (count, lo, hi, key))
    return [hi] + ([lo] if count > 1 else []) + [r.randint(lo, hi) for _ in range(count - 2)]


def _lengths(case):
    """[(cached tokens after the call, new tokens)] of a place case's sequences."""
    new = sorted(_spread(case["B"], case["min_n"], case["max_n"], "new"))
    return [(max(n, m), m) for n, m in zip(sorted(_spread(case["B"], case["min_len"], case["max_len"], "len")), new)]


def _deal(case):
    """[(adapter, rows)] of a lora case: single rows of a step, runs of a prompt; -1: no adapter."""
    M, L, none = case["M"], case["adapters"], case["none"]
    if case["rows"] == "step":
        return [(-1, 1)] * none + [(i % L, 1) for i in range(M - none)]
    cuts = sorted(_spread(L - 1, 1, M - none - 1, "cut")) if L > 1 else []
    at = [0] + cuts + [M - none]
    return ([(-1, none)] if none else []) + [(i, at[i + 1] - at[i]) for i in range(L) if at[i + 1] > at[i]]


def _ranks(case):
    """The rank of each adapter; the pool's is the largest."""
    if not case["ragged"]:
        return [case["rank"]] * case["adapters"]
    return _spread(case["adapters"], max(1, case["rank"] // 4), case["rank"], "rank")


def work(case):
    if case["op"] == "norm":
        n = case["M"] * case["K"]
        x = SIZE[case["x"]]
        b = n * (x * (3 if case["res"] else 1) + SIZE[case["out"]]) + 4 * case["K"]
        if case["out"] == "int8":
            b += 4 * case["M"] + 4 * n + n  # the scales, and the values that the codes stand for, read back
        return {"bytes": b, "flops": 5 * n}
    if case["op"] == "rope":
        n = case["T"] * case["heads"] * case["d"]
        return {"bytes": 2 * n * SIZE[case["x"]] + 4 * case["T"], "flops": 3 * case["T"] * case["heads"] * case["rot"]}
    if case["op"] == "place":
        rows = sum(m for _, m in _lengths(case))
        kv = 2 * rows * case["hkv"] * case["d"]
        q = rows * case["hq"] * case["d"]
        cached = kv * SIZE[case["kv"]] + (4 * kv // case["d"] if case["kv"] == "int8" else 0)
        back = cached + 4 * kv if case["kv"] == "int8" else 0
        return {"bytes": (2 * q + kv) * SIZE[case["x"]] + cached + back, "flops": 3 * (q + kv // 2)}
    used = {}
    for a, n in _deal(case):
        if a >= 0:
            used[a] = used.get(a, 0) + n
    ranks, K, N = _ranks(case), case["K"], case["N"]
    rows = sum(used.values())
    return {"bytes": rows * (K * SIZE[case["x"]] + 8 * N) + sum(2 * ranks[a] * (K + N) for a in used) + 4 * case["M"],
            "flops": sum(2 * n * ranks[a] * (K + N) for a, n in used.items())}


# ------------------------------------------------------------------ inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


CONTEXT, FAST, SLOW = 4096, 32.0, 1.0  # the trained context of the stretched frequencies and the bounds of their ramp, in turns


def _frequencies(rot, base, scaling, factor):
    """(turns a token of each pair, factor of the rotated values)."""
    if scaling == "ntk":
        base = base * math.pow(factor, rot / (rot - 2.0)) if rot > 2 else base
    half = rot // 2
    f = [math.pow(base, -2.0 * i / rot) / (2.0 * math.pi) for i in range(half)]
    if scaling == "linear":
        return [v / factor for v in f], 1.0
    if scaling == "yarn":
        at = [rot * math.log(CONTEXT / (2.0 * math.pi * turns)) / (2.0 * math.log(base)) for turns in (FAST, SLOW)]
        low, high = max(math.floor(at[0]), 0.0), min(math.ceil(at[1]), rot - 1.0)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(half)]
        return [v / factor * g + v * (1.0 - g) for v, g in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    if scaling == "bands":
        keep = [min(max((CONTEXT * v - SLOW) / (4.0 - SLOW), 0.0), 1.0) for v in f]
        return [v * g + v / factor * (1.0 - g) for v, g in zip(f, keep)], 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 29)
    rnd = random.Random("%d %s" % (seed, case["op"]))
    s = dict(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        x = normal(M, K)
        x[:, rnd.randrange(K)] *= 50  # a channel that stands out, as activations have
        s["xv"] = x.to(TYPES[case["x"]])
        s["rv"] = (3 * normal(M, K)).to(TYPES[case["x"]]) if case["res"] else None
        s["w"] = 0.2 * normal(K) + (1.0 - case["offset"])
        return s
    if case["op"] == "lora":
        M, K, N, r, L = (case[k] for k in ("M", "K", "N", "rank", "adapters"))
        deal = _deal(case)
        names = list(range(L))
        rnd.shuffle(names)  # which adapter of the pool a dealt one is: ranks go with it
        rnd.shuffle(deal)
        s["ids"] = _ints([-1 if a < 0 else names[a] for a, n in deal for _ in range(n)])
        ranks = [0] * L
        for a, v in enumerate(_ranks(case)):
            ranks[names[a]] = v
        s["ranks"] = _ints(ranks) if case["ragged"] else None
        s["xv"] = normal(M, K).to(TYPES[case["x"]])
        s["A"] = (normal(L, r, K) * K ** -0.5).to(torch.bfloat16)
        s["B"] = (normal(L, N, r) * 0.3).to(torch.bfloat16)
        s["scales"] = 0.5 + 2 * torch.rand((L,), generator=g, device=DEV)
        s["y"] = normal(M, N)
        if own:
            import int4_weight_quantized_amd as w4

            s["work"] = torch.empty(w4.lora_workspace_bytes(M, K, N, r), dtype=torch.uint8, device=DEV)
        return s
    freqs, s["mag"] = _frequencies(case["rot"], 10000.0, case["scaling"], case["factor"])
    s["freqs"] = torch.tensor(freqs, dtype=torch.float64, device=DEV)
    dt = TYPES[case["x"]]
    if case["op"] == "rope":
        T = case["T"]
        s["xv"] = normal(T, case["row"], case["d"]).to(dt)[:, :case["heads"]]
        cuts = sorted(rnd.randrange(T) for _ in range(min(T - 1, 3)))
        ends = cuts + [T]
        begin = [rnd.randrange(case["far"]) for _ in ends]
        s["pos"] = torch.cat([torch.arange(b, b + e - a, dtype=torch.int32, device=DEV) for a, e, b in zip([0] + cuts, ends, begin)])
    else:
        ps, hq, hkv, d = case["ps"], case["hq"], case["hkv"], case["d"]
        deal = _lengths(case)
        rnd.shuffle(deal)
        need = [-(-n // ps) for n, _ in deal]
        W, pages = max(need) + 1, sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        at = _ints([sum(need[:i]) for i in range(len(need))])[:, None] + torch.arange(W, device=DEV, dtype=torch.int32)
        s["table"] = torch.where(torch.arange(W, device=DEV) < _ints(need)[:, None], order[at.clamp(max=pages - 1).long()],
                                 -1).to(torch.int32).contiguous()
        new = [m for _, m in deal]
        cu = [sum(new[:i]) for i in range(len(new) + 1)]
        s["cu"] = _ints(cu)
        s["rows"] = cu[-1]
        s["start"] = _ints([n - m for n, m in deal])
        shape = (1, pages, hkv, ps, d)
        s["k"], s["v"] = (torch.zeros(shape, dtype=TYPES[case["kv"]], device=DEV) for _ in range(2))
        s["ks"], s["vs"] = (torch.zeros(shape[:4], device=DEV) if case["kv"] == "int8" else None for _ in range(2))
        joint = normal(cu[-1], hq + 2 * hkv, d).to(dt)
        s["xq"], s["xk"], s["xv"] = joint[:, :hq], joint[:, hq:hq + hkv], joint[:, hq + hkv:]
    if own:
        import int4_weight_quantized_amd as w4

        s["rope"] = w4.Rope(case["rot"], base=10000.0, layout=case["layout"], scaling=case["scaling"], factor=case["factor"],
                            context=CONTEXT, fast=4.0 if case["scaling"] == "bands" else FAST, slow=SLOW, device=DEV)
        if case["op"] == "place":
            s["cache"] = w4.KVCache(s["k"], s["v"], s["ks"], s["vs"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import int4_weight_quantized_amd as w4

    op = s["op"]
    if op == "norm":
        if s["out"] == "int8":
            q, sx, h = w4.a8_rms_norm(s["xv"], s["w"], s["eps"], residual=s["rv"], offset=s["offset"])
            return {"y": torch.mul(q, sx[:, None]), "sx": sx, "sum": h}  # the values that the codes stand for
        y, h = w4.rms_norm(s["xv"], s["w"], s["eps"], residual=s["rv"], offset=s["offset"], dtype=TYPES[s["out"]])
        return {"y": y, "sum": h}
    if op == "rope":
        return w4.rope_rotate(s["xv"], s["pos"], s["rope"])
    if op == "place":
        q = w4.kv_append_rope(s["cache"], 0, s["xq"], s["xk"], s["xv"], s["table"], s["start"], s["rope"], s["cu"])
        if s["ks"] is None:
            return {"q": q, "k": s["k"], "v": s["v"]}
        k, v = w4.kv_gather(s["cache"], 0, s["table"], s["start"], s["cu"], s["rows"])
        return {"q": q, "k": k, "v": v, "ks": s["ks"], "vs": s["vs"]}
    return w4.lora_add(s["y"], s["xv"], s["ids"], s["A"], s["B"], scales=s["scales"], ranks=s["ranks"], workspace=s["work"])


def _run_plain(s):
    return {"norm": _plain_norm, "rope": _plain_rope, "place": _plain_place, "lora": _plain_lora}[s["op"]](s)


def _plain_norm(s):
    """The mean is taken in 64 bits and rounded once, as quotients are: codes lie next to a border otherwise."""
    h = s["xv"].float()
    if s["rv"] is not None:
        h = h + s["rv"].float()
    r = (1.0 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + s["eps"])).float()
    y = (h * r) * (s["w"] + s["offset"])
    total = h.to(TYPES[s["x"]]) if s["rv"] is not None else None
    if s["out"] != "int8":
        return {"y": y.to(TYPES[s["out"]]), "sum": total}
    sx = (y.abs().amax(-1).double() / 127).float()
    code = torch.round((y.double() / sx.double()[:, None]).float()).clamp(-128, 127)
    return {"y": torch.where(sx[:, None] > 0, code, 0.0) * sx[:, None], "sx": sx, "sum": total}


def _turned(x, pos, s):
    """x [T, heads, d] rotated to positions pos [T], in 32 bits; angles in 64."""
    rot, half = s["rot"], s["rot"] // 2
    turns = pos.double()[:, None] * s["freqs"]
    angle = 2 * math.pi * (turns - torch.round(turns))
    c, n = ((f(angle) * s["mag"]).float()[:, None] for f in (torch.cos, torch.sin))
    y = x.float().clone()
    if s["layout"] == "half":
        a, b = y[..., :half].clone(), y[..., half:rot].clone()
        y[..., :half], y[..., half:rot] = a * c - b * n, b * c + a * n
    else:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * n, b * c + a * n
    return y


def _plain_rope(s):
    return _turned(s["xv"], s["pos"], s).to(s["xv"].dtype)


def _plain_place(s):
    row = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(s["cu"][1:].contiguous().long(), row, right=True)
    p = s["start"].long()[b] + row - s["cu"].long()[b]
    page, slot = s["table"].long()[b, p // s["ps"]], p % s["ps"]
    q = _turned(s["xq"], p, s).to(s["xq"].dtype)
    k, v = _turned(s["xk"], p, s), s["xv"].float()
    if s["ks"] is None:
        s["k"][0][page, :, slot] = k.to(torch.bfloat16)
        s["v"][0][page, :, slot] = v.to(torch.bfloat16)
        return {"q": q, "k": s["k"], "v": s["v"]}
    return {"q": q, "k": _plain_quantize(k, s["k"][0], s["ks"][0], page, slot),
            "v": _plain_quantize(v, s["v"][0], s["vs"][0], page, slot), "ks": s["ks"], "vs": s["vs"]}


def _plain_quantize(x, codes, scales, page, slot):
    sc = x.abs().amax(-1) * torch.full((), 1.0 / 127, device=DEV)  # the cache's rule: one multiplication
    c = torch.where(sc[..., None] > 0, torch.round(x / sc[..., None]).clamp(-128, 127), 0.0)
    codes[page, :, slot] = c.to(torch.int8)
    scales[page, :, slot] = sc
    return codes[page, :, slot].float() * scales[page, :, slot][..., None]


def _plain_lora(s):
    """Every row against every adapter, the others' results dropped, so that two products do it."""
    L, r, K = s["A"].shape
    low = torch.matmul(s["xv"].float(), s["A"].float().view(L * r, K).T).view(-1, L, r)
    take = (s["ids"][:, None] == torch.arange(L, device=DEV))[..., None]
    if s["ranks"] is not None:
        take = take & (torch.arange(r, device=DEV) < s["ranks"][:, None])
    low = torch.where(take, low * s["scales"][:, None], 0.0)
    s["y"] += torch.matmul(low.view(-1, L * r), s["B"].float().transpose(1, 2).reshape(L * r, -1))
    return s["y"]


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    if case["op"] == "norm":
        h = s["xv"].double() if s["rv"] is None else s["xv"].double() + s["rv"].double()
        y = h * torch.rsqrt((h * h).sum(1) / case["K"] + case["eps"])[:, None] * (case["offset"] + s["w"].double())
        total = None if s["rv"] is None else h
        if case["out"] == "int8":
            return {"y": None, "sx": y.abs().max(1).values / 127, "sum": total}  # a code on a tie may fall to either side
        return {"y": y, "sum": total}
    if case["op"] == "lora":
        out = s["y"].double()
        ranks = [case["rank"]] * case["adapters"] if s["ranks"] is None else s["ranks"].tolist()
        for a in sorted(set(s["ids"].tolist()) - {-1}):
            rows = torch.nonzero(s["ids"] == a)[:, 0]
            low = s["xv"][rows].double() @ s["A"][a, :ranks[a]].double().T
            out[rows] += float(s["scales"][a]) * (low @ s["B"][a, :, :ranks[a]].double().T)
        return out

    def turned(x, pos):
        """Pairs as complex numbers times a unit of the angle."""
        rot, half = case["rot"], case["rot"] // 2
        unit = torch.polar(torch.full((len(pos), half), s["mag"], dtype=torch.float64, device=DEV),
                           torch.fmod(pos.double()[:, None] * s["freqs"], 1.0) * (2 * math.pi))[:, None]
        x = x.double()
        head, rest = x[..., :rot], x[..., rot:]
        pairs = head.unflatten(-1, (2, half)).transpose(-1, -2) if case["layout"] == "half" else head.unflatten(-1, (half, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
        return torch.cat([(z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2), rest], -1)

    if case["op"] == "rope":
        return turned(s["xv"], s["pos"])
    table, start, cu = s["table"].tolist(), s["start"].tolist(), s["cu"].tolist()
    pos = [p for b in range(len(start)) for p in range(start[b], start[b] + cu[b + 1] - cu[b])]
    where = [(table[b][p // case["ps"]], p % case["ps"]) for b in range(len(start))
             for p in range(start[b], start[b] + cu[b + 1] - cu[b])]
    pos = torch.tensor(pos, device=DEV)
    page, slot = (torch.tensor(x, device=DEV) for x in zip(*where))
    out = {"q": turned(s["xq"], pos)}
    for name, x in (("k", turned(s["xk"], pos)), ("v", s["xv"].double())):
        if s["ks"] is None:
            out[name] = s[name].double()
            out[name][0][page, :, slot] = x
        else:
            out[name] = None  # a code on a tie may fall to either side
            out[name + "s"] = s[name + "s"].double()
            out[name + "s"][0][page, :, slot] = x.abs().max(-1).values / 127
    return out
