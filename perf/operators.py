"""The operators for weights that depend on the token, and what they are measured on.

Four operators of a serving step: the router (top-k gate and the sort of the
chosen (token, expert) entries into one segment per expert), the linear layer
grouped by expert on separated-quantization weights, the weighted sum of each
token's expert rows, and the low-rank adapters of many requests beside a shared
projection.  `run` computes them in plain torch operations, or, where `own` is
true, by the calls of the package.
"""
import math

import torch

own = False

G = 128  # channels per residual group and per weight tile


def _up(a, b):
    return -(-a // b) * b


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # one decode step's router: 16 sequences, 64 experts, 4 chosen
        dict(name="route_decode", op="route", T=16, E=64, k=4, gate="topk", ties=False),
        # the router over a long batch of prompts; logits on a coarse grid, so that ties are met
        dict(name="route_prefill", op="route", T=8192, E=128, k=8, gate="all", ties=True),
        # one sequence decoding through 2 of 8 wide experts: two experts' weights are streamed
        dict(name="grouped_one_token", op="grouped", T=1, E=8, k=2, N=14336, K=4096, n_out=20, mask=0, skew=0.0, sorted=False),
        # the down projection of a decode batch of 16: rows already in expert order
        dict(name="grouped_decode_down", op="grouped", T=16, E=8, k=2, N=4096, K=14336, n_out=72, mask=0, skew=0.0, sorted=True),
        # a mixed batch (decode and short prompts) over many experts, ragged, threshold trunk, odd sizes
        dict(name="grouped_ragged", op="grouped", T=203, E=16, k=4, N=4090, K=4000, n_out=21, mask=60, skew=1.0, sorted=False),
        # a batch of prompts: 4096 entries over 8 experts
        dict(name="grouped_prefill", op="grouped", T=2048, E=8, k=2, N=14336, K=4096, n_out=20, mask=0, skew=0.5, sorted=False),
        # the expert rows of a decode batch summed into the residual stream
        dict(name="combine_decode", op="combine", T=16, k=2, N=4096, drop=0.0, base=True),
        # the same for a batch of prompts, with entries that were dropped
        dict(name="combine_prefill", op="combine", T=4099, k=4, N=4096, drop=0.1, base=False),
        # one request with an adapter
        dict(name="lora_one_token", op="lora", M=1, S=8, R=16, K=4096, N=4096, dtype="bf16", none=0.0, ld=4096, ragged=False),
        # a decode batch of 64 requests over 32 adapters of mixed rank, on the fused qkv projection
        dict(name="lora_decode", op="lora", M=64, S=32, R=64, K=4096, N=12288, dtype="bf16", none=0.1, ld=12288, ragged=True),
        # binary32 adapters on a slice of a wider projection; odd row count
        dict(name="lora_mixed_f32", op="lora", M=333, S=5, R=24, K=11008, N=4096, dtype="f32", none=0.3, ld=12288, ragged=True),
        # prompts of several requests, binary16 adapters
        dict(name="lora_prefill", op="lora", M=2048, S=8, R=64, K=4096, N=14336, dtype="f16", none=0.0, ld=14336, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "grouped", "grouped", "grouped", "combine", "lora", "lora", "lora"])
    if op == "route":
        E = _log(rng, 4, 256)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)), gate=rng.choice(["topk", "all"]),
                    ties=rng.random() < 0.5)
    if op == "combine":
        return dict(op=op, T=_log(rng, 1, 4096), k=rng.randint(1, 4), N=_log(rng, 64, 4096), drop=rng.choice([0.0, 0.2]),
                    base=rng.random() < 0.5)
    if op == "grouped":
        while True:
            E, N, K, T = _log(rng, 2, 64), _log(rng, 128, 14336), _log(rng, 128, 14336), _log(rng, 1, 2048)
            k = rng.randint(1, min(4, E))
            if E * N * K <= 8 * 14336 * 4096 and T * k * N * K <= 4096 * 14336 * 4096 and T * k * K <= 4096 * 14336:
                break
        return dict(op=op, T=T, E=E, k=k, N=N, K=K, n_out=rng.randint(0, 64), mask=rng.choice([0, 0, 50, 70]),
                    skew=rng.choice([0.0, 0.5, 1.0]), sorted=rng.random() < 0.5)
    M, S, R = _log(rng, 1, 2048), _log(rng, 1, 32), _log(rng, 4, 128)
    K, N = _log(rng, 128, 14336), _log(rng, 128, 14336)
    return dict(op=op, M=M, S=S, R=R, K=K, N=N, dtype=rng.choice(["bf16", "f16", "f32"]), none=rng.choice([0.0, 0.3]),
                ld=N + rng.choice([0, 0, 128]), ragged=rng.random() < 0.5)


def _active(c):
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])


def work(case):
    c = case
    if c["op"] == "route":
        n = c["T"] * c["k"]
        return {"bytes": 4 * c["T"] * c["E"] + 16 * n + 4 * (c["E"] + 1), "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "combine":
        n = c["T"] * c["k"] * (1 - c["drop"])
        return {"bytes": 4 * c["N"] * (n + c["T"] * (2 if c["base"] else 1)) + 8 * c["T"] * c["k"], "flops": 2 * n * c["N"]}
    if c["op"] == "grouped":
        n = c["T"] * c["k"]
        planes = 2 if c["mask"] else 1
        weight = c["N"] * (c["K"] + planes * c["K"] / 8 + 4 * -(-c["K"] // G) + 4)
        rows = n if c["sorted"] else c["T"]
        return {"bytes": _active(c) * weight + rows * (c["K"] + 4 + 4 * c["n_out"]) + 4 * n * c["N"] + 4 * (c["E"] + 1),
                "flops": 2 * n * c["N"] * c["K"]}
    size = 4 if c["dtype"] == "f32" else 2
    used = c["S"] * (1 - (1 - (1 - c["none"]) / c["S"]) ** c["M"])
    rank = c["R"] * (0.75 if c["ragged"] else 1.0)
    live = c["M"] * (1 - c["none"])
    return {"bytes": 4 * live * c["K"] + 8 * c["M"] * c["N"] + used * rank * (c["K"] + c["N"]) * size + 4 * c["M"],
            "flops": 2 * live * rank * (c["K"] + c["N"])}


# ---- inputs --------------------------------------------------------------------

def _half_away(v):
    return torch.where(v < 0, -(0.5 - v).floor(), (v + 0.5).floor())


def _expert(case, gen):
    """One expert's weight, split and packed as a program that serves it keeps it:
    sign (and mask) bits, row scales, residual codes and group scales, in tiles
    of 16 rows x 128 channels."""
    N, K = case["N"], case["K"]
    rows, cols = _up(N, 16), _up(K, G)
    u = torch.rand(N, K, generator=gen, device="cuda")
    W = 0.02 * torch.sign(u - 0.5) * -torch.log1p(-2 * (u - 0.5).abs().clamp(max=0.4999999))
    A = W.abs()
    if case["mask"]:
        at = max(1, -(-case["mask"] * K // 100)) - 1
        keep = A > torch.sort(A, dim=1).values[:, at:at + 1]
    else:
        keep = torch.ones_like(A, dtype=torch.bool)
    alpha = ((A.double() * keep).sum(1) / keep.sum(1).clamp(min=1)).float()
    sign = W >= 0
    res = W.double() - torch.where(keep, torch.where(sign, 1.0, -1.0), 0.0).double() * alpha.double()[:, None]
    full = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    full[:N, :K] = res
    grp = full.view(rows, cols // G, G)
    scale = (grp.abs().amax(2) / 127).float()
    codes = torch.where(scale[..., None] > 0, _half_away(grp / scale.double()[..., None]), 0.0).clamp(-127, 127).to(torch.int8)
    rb, g = rows // 16, cols // G
    codes = codes.view(rb, 2, 8, g, 4, 4, 2, 4).permute(0, 3, 2, 4, 5, 6, 1, 7).reshape(rows, cols).contiguous()
    place = (1 << (8 * torch.arange(4, device="cuda")[None, :] + torch.arange(8, device="cuda")[:, None])).to(torch.int64)

    def bits(b):
        wide = torch.zeros(rows, cols, dtype=torch.bool, device="cuda")
        wide[:N, :K] = b
        w = (wide.view(rb, 2, 8, g, 4, 8, 4) * place).sum((5, 6)).to(torch.int32)  # wraps to the word's bits
        return w.permute(0, 3, 2, 4, 1).reshape(rows, cols // 32).contiguous()

    al = torch.zeros(rows, device="cuda")
    al[:N] = alpha
    sc = scale.view(rb, 16, g).permute(0, 2, 1).reshape(rows, g).contiguous()
    return bits(sign), (bits(keep) if case["mask"] else None), al, codes, sc


def _grouped(case, gen):
    T, E, k, K, n_out = case["T"], case["E"], case["k"], case["K"], case["n_out"]
    parts = [_expert(case, gen) for _ in range(E)]
    sign, mask, alpha, codes, scale = (None if p[0] is None else torch.cat(p) for p in zip(*parts))
    pref = torch.randn(T, E, generator=gen, device="cuda") + case["skew"] * torch.linspace(1, -1, E, device="cuda")
    ids = torch.topk(pref, k, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    offsets = torch.searchsorted(ids[order].contiguous(), torch.arange(E + 1, device="cuda")).to(torch.int32)
    rows = T * k if case["sorted"] else T
    x = torch.randn(rows, K, generator=gen, device="cuda")
    idx = torch.randperm(K, generator=gen, device="cuda")[:min(n_out, K)].sort().values
    x[:, idx] *= 30
    rest = x.clone()
    rest[:, idx] = 0
    sx = (rest.abs().amax(1).double() / 127).float()
    xq = torch.zeros(rows, _up(K, G), dtype=torch.int8, device="cuda")
    xq[:, :K] = _half_away(rest.double() / sx.double().clamp(min=1e-300)[:, None]).clamp(-127, 127).to(torch.int8)
    cap = int((offsets[1:] - offsets[:-1]).max())
    return dict(sign=sign, mask=mask, alpha=alpha, codes=codes, scale=scale, xq=xq, sx=sx, idx=idx.to(torch.int32),
                x_out=x[:, idx].contiguous(), offsets=offsets, cap=cap,
                order=None if case["sorted"] else order.to(torch.int32))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    if c["op"] == "route":
        logits = 2 * torch.randn(c["T"], c["E"], generator=gen, device="cuda")
        if c["ties"]:
            logits = (logits * 8).round() / 8
        return dict(case=c, logits=logits)
    if c["op"] == "combine":
        n = c["T"] * c["k"]
        place = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
        place = torch.where(torch.rand(n, generator=gen, device="cuda") < c["drop"], -1, place).view(c["T"], c["k"])
        gates = torch.softmax(torch.randn(c["T"], c["k"], generator=gen, device="cuda"), 1)
        return dict(case=c, place=place.contiguous(), gates=gates, z=torch.randn(n, c["N"], generator=gen, device="cuda"),
                    base=torch.randn(c["T"], c["N"], generator=gen, device="cuda") if c["base"] else None)
    if c["op"] == "grouped":
        return dict(case=c, **_grouped(c, gen))
    M, S, R = c["M"], c["S"], c["R"]
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[c["dtype"]]
    A = (torch.randn(S, R, c["K"], generator=gen, device="cuda") / math.sqrt(c["K"])).to(dt)
    B = (0.05 * torch.randn(S, c["N"], R, generator=gen, device="cuda")).to(dt)
    ids = torch.randint(S, (M,), generator=gen, device="cuda")
    if M > 256:  # prompts: the tokens of a request lie together
        ids = ids[torch.arange(M, device="cuda") // 97 * 97]
    ids = torch.where(torch.rand(M, generator=gen, device="cuda") < c["none"], -1, ids).to(torch.int32)
    rank = torch.randint((R + 1) // 2, R + 1, (S,), generator=gen, device="cuda") if c["ragged"] else torch.full((S,), R, device="cuda")
    x = torch.randn(M, c["K"], generator=gen, device="cuda")
    wide = torch.randn(M, c["ld"], generator=gen, device="cuda")
    return dict(case=c, A=A, B=B, ids=ids, rank=rank.to(torch.int32), x=x, base=wide[:, c["ld"] - c["N"]:],
                scale=0.5 + torch.rand(S, generator=gen, device="cuda"))


# ---- the operators ---------------------------------------------------------------

def _plain_route(c, logits):
    value, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    value, ids = value[:, :c["k"]], ids[:, :c["k"]]
    top = value[:, :1]
    over = value if c["gate"] == "topk" else logits
    gates = torch.exp(value - top) / torch.exp(over - top).sum(1, keepdim=True)
    flat = ids.reshape(-1)
    by, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(by, torch.arange(c["E"] + 1, device="cuda"))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    i32 = torch.int32
    return dict(ids=ids.to(i32), gates=gates, offsets=offsets.to(i32), order=order.to(i32), place=place.view_as(ids).to(i32))


def _plain_weights(s, which):
    """Binary32 weights [len(which)][rows][channels] of the experts `which`."""
    c = s["case"]
    rows, cols = _up(c["N"], 16), _up(c["K"], G)
    rb, g, n = rows // 16, cols // G, which.numel()
    q = s["codes"].view(c["E"], -1)[which].view(n, rb, g, 8, 4, 4, 2, 2, 4).permute(0, 1, 7, 3, 2, 4, 5, 6, 8).reshape(n, rows, g, G)
    at = 8 * torch.arange(4, device="cuda", dtype=torch.int32)[None, :] + torch.arange(8, device="cuda", dtype=torch.int32)[:, None]

    def bits(words):
        w = words.view(c["E"], -1)[which].view(n, rb, g, 8, 4, 2, 1, 1)
        return ((w >> at) & 1).permute(0, 1, 5, 3, 2, 4, 6, 7).reshape(n, rows, cols)

    trunk = (2 * bits(s["sign"]) - 1).float() * s["alpha"].view(c["E"], rows, 1)[which]
    if s["mask"] is not None:
        trunk = trunk * bits(s["mask"])
    scale = s["scale"].view(c["E"], rb, g, 16)[which].permute(0, 1, 3, 2).reshape(n, rows, g, 1)
    w = trunk + (q.float() * scale).view(n, rows, cols)
    return w[:, :c["N"], :c["K"]]


def _plain_grouped(s):
    c = s["case"]
    x = s["xq"][:, :c["K"]].float() * s["sx"][:, None]
    x[:, s["idx"].long()] = s["x_out"]
    if s["order"] is not None:
        x = x[(s["order"] // c["k"]).long()]
    n = x.shape[0]
    offsets = s["offsets"].long()
    expert = torch.searchsorted(offsets[1:], torch.arange(n, device="cuda"), right=True)
    if n <= c["E"]:  # few entries: the weight of each entry
        return torch.bmm(_plain_weights(s, expert), x[:, :, None])[:, :, 0]
    slot = torch.arange(n, device="cuda") - offsets[expert]
    padded = torch.zeros(c["E"], s["cap"], c["K"], device="cuda")
    padded[expert, slot] = x
    y = torch.bmm(padded, _plain_weights(s, torch.arange(c["E"], device="cuda")).transpose(1, 2))
    return y[expert, slot]


def _plain_combine(s):
    live = s["place"] >= 0
    rows = s["z"][s["place"].clamp(min=0).long()]
    out = (rows * torch.where(live, s["gates"], 0.0)[..., None]).sum(1)
    return out if s["base"] is None else out + s["base"]


def _plain_lora(s):
    c = s["case"]
    S, R = c["S"], c["R"]
    v = (s["x"] @ s["A"].float().view(S * R, c["K"]).t()).view(c["M"], S, R)
    slots = torch.arange(S, device="cuda")
    live = (s["ids"][:, None] == slots)[:, :, None] & (torch.arange(R, device="cuda") < s["rank"][:, None])
    v = torch.where(live, v, 0.0) * s["scale"][:, None]
    return s["base"] + v.view(c["M"], S * R) @ s["B"].float().permute(0, 2, 1).reshape(S * R, c["N"])


def run(state):
    s, c = state, state["case"]
    if own:
        import decode_matvec_sq_b200 as sq
        if c["op"] == "route":
            r = sq.route(s["logits"], c["k"], gate=c["gate"])
            return dict(ids=r.ids, gates=r.gates, offsets=r.offsets, order=r.order, place=r.place)
        if c["op"] == "combine":
            return sq.combine(s["z"], s["gates"], s["place"], base=s["base"])
        if c["op"] == "grouped":
            if "experts" not in s:  # the handle and the workspace that a serving program keeps
                s["experts"] = sq.experts_from_arrays(c["E"], c["N"], c["K"], s["sign"], s["alpha"], s["codes"], s["scale"],
                                                      mask_bits=s["mask"])
                s["workspace"] = sq.new_grouped_workspace(s["experts"], c["T"] * c["k"])
            return sq.grouped_linear(s["experts"], s["xq"], s["sx"], s["x_out"], s["idx"], s["offsets"], order=s["order"],
                                     div=c["k"] if s["order"] is not None else 1, workspace=s["workspace"])
        if "bank" not in s:
            s["bank"] = sq.LoraBank(s["A"], s["B"], s["scale"], s["rank"])
            s["workspace"] = sq.new_lora_workspace(s["bank"], c["M"])
        return sq.lora_add(s["bank"], s["x"], s["ids"], s["base"], workspace=s["workspace"])
    if c["op"] == "route":
        return _plain_route(c, s["logits"])
    if c["op"] == "combine":
        return _plain_combine(s)
    if c["op"] == "grouped":
        return _plain_grouped(s)
    return _plain_lora(s)


# ---- the definition in 64 bits -------------------------------------------------------

def _exact_route(c, logits):
    l = logits.double()
    i = torch.arange(c["E"], device="cuda")
    gates, ids, left = [], [], l.clone()
    for _ in range(c["k"]):  # the largest of what is left, the lowest index among equals
        m = left.amax(1, keepdim=True)
        j = torch.where(left == m, i, c["E"]).amin(1)
        ids.append(j)
        left[torch.arange(c["T"], device="cuda"), j] = -math.inf
    ids = torch.stack(ids, 1)
    v = l.gather(1, ids)
    z = torch.logsumexp(v if c["gate"] == "topk" else l, 1, keepdim=True)
    gates = torch.exp(v - z)
    key = ids.reshape(-1) * (c["T"] * c["k"]) + torch.arange(c["T"] * c["k"], device="cuda")
    order = torch.argsort(key)
    place = torch.argsort(order)
    offsets = torch.tensor([0] + torch.bincount(ids.reshape(-1), minlength=c["E"]).cumsum(0).tolist(), device="cuda")
    i32 = torch.int32
    return dict(ids=ids.to(i32), gates=gates, offsets=offsets.to(i32), order=order.to(i32), place=place.view_as(ids).to(i32))


def _exact_grouped(s):
    c = s["case"]
    N, K, rows, cols = c["N"], c["K"], _up(c["N"], 16), _up(c["K"], G)
    r, j = torch.arange(N, device="cuda")[:, None], torch.arange(K, device="cuda")[None, :]
    tile = (r // 16) * (cols // G) + j // G
    lane = (r % 8) * 4 + (j % G) // 32
    w = (j % 32) // 4
    code_at = (tile * 32 + lane) * 64 + w // 2 * 16 + (w % 2 * 2 + r % 16 // 8) * 4 + j % 4
    word_at = (tile * 32 + lane) * 2 + r % 16 // 8
    bit = 8 * (j % 4) + w
    scale_at = tile * 16 + r % 16
    x = s["xq"][:, :K].double() * s["sx"].double()[:, None]
    x[:, s["idx"].long()] = s["x_out"].double()
    bounds = s["offsets"].tolist()
    y = torch.zeros(bounds[-1], N, dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        codes = s["codes"].view(c["E"], -1)[e][code_at].double()
        W = codes * s["scale"].view(c["E"], -1)[e][scale_at].double()
        sgn = ((s["sign"].view(c["E"], -1)[e][word_at] >> bit) & 1).double() * 2 - 1
        if s["mask"] is not None:
            sgn = sgn * ((s["mask"].view(c["E"], -1)[e][word_at] >> bit) & 1)
        W += sgn * s["alpha"].view(c["E"], rows)[e, :N, None].double()
        src = torch.arange(a, b, device="cuda") if s["order"] is None else (s["order"][a:b] // c["k"]).long()
        y[a:b] = x[src] @ W.t()
    return y


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "route":
        return _exact_route(c, s["logits"])
    if c["op"] == "combine":
        out = torch.zeros(c["T"], c["N"], dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            p = s["place"][:, j].long()
            out += torch.where(p >= 0, s["gates"][:, j].double(), 0.0)[:, None] * s["z"][p.clamp(min=0)].double()
        return out if s["base"] is None else out + s["base"].double()
    if c["op"] == "grouped":
        return _exact_grouped(s)
    y = s["base"].double().clone()
    for a, r in enumerate(s["rank"].tolist()):
        t = (s["ids"] == a).nonzero()[:, 0]
        y[t] += s["scale"][a].double() * (s["x"][t].double() @ s["A"][a, :r].double().t()) @ s["B"][a, :, :r].double().t()
    return y
