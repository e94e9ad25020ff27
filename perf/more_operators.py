"""Routing by scores and groups, and the experts' products in 8-bit floating point:
their cases, plain forms and exact values.

Operators: select (select_experts: softmax or sigmoid scores of given logits, a
balance bias on the choice, groups, top-k, weights); up and down (the grouped gated
product and the grouped product with the weighted sum, on E4M3 codes with one scale
per 128 values of an activation and per 128 x 128 block of a weight); ffn (both, the
activations between them quantised by the first); quantize (bf16 to such codes and
back). A routed slot i = t * width + s; w13 holds every expert's I gate rows, then
its I up rows, and its scales those of the gate rows' blocks, then the up rows'.
"""
import math

import torch

own = False

BLOCK = 128                             # values that share a scale
LARGE = 16384 * 8 * 2048 * 768          # slots x H x I of the largest case
WEIGHTS = 513 * 512 * 4096              # experts x H x I of the largest weights


def _ffn(name, op, T, H, E, S, k, I, A, zipf=0.0):
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "S": S, "k": k, "I": I, "A": A, "zipf": zipf}


def _sel(name, T, E, S, k, scoring, bias, groups, kept, best, dtype, renorm):
    return {"name": name, "op": "select", "T": T, "E": E, "S": S, "k": k, "scoring": scoring, "bias": bias, "groups": groups,
            "kept": kept, "best": best, "dtype": dtype, "renorm": renorm}


def listed():
    return [
        # speculative verify step: sigmoid scores with a balance bias, one group, the shared slot
        _sel("select_verify_4", 4, 512, 1, 10, "sigmoid", True, 1, 1, 1, "fp32", True),
        # odd-sized prompt: 8 groups by their two best, 4 of them kept, bf16 logits
        _sel("select_groups_2047", 2047, 256, 0, 8, "sigmoid", True, 8, 4, 2, "bf16", True),
        # large prefill batch: softmax scores, groups by their best, weights not renormalised
        _sel("select_large_16384", 16384, 512, 1, 10, "softmax", False, 8, 3, 1, "fp32", False),
        # speculative verify step: latency, weights streamed
        _ffn("up_verify_4", "up", 4, 4096, 512, 1, 10, 512, 64),
        # large prefill batch: about 1024 rows an expert
        _ffn("up_large_16384", "up", 16384, 2048, 128, 0, 8, 768, 128),
        # one sequence decoding one token: the smallest call
        _ffn("down_token_1", "down", 1, 2048, 128, 0, 8, 768, 64),
        # odd-sized prompt, skewed: ragged segments
        _ffn("down_skewed_2047", "down", 2047, 2048, 128, 0, 8, 768, 128, 1.1),
        # both products: a decode batch, a short prompt with a few hot experts, a large batch
        _ffn("ffn_decode_8", "ffn", 8, 4096, 512, 1, 10, 512, 64),
        _ffn("ffn_skewed_512", "ffn", 512, 2048, 128, 0, 8, 768, 64, 1.1),
        _ffn("ffn_large_16384", "ffn", 16384, 2048, 128, 0, 8, 768, 128),
        # hidden states of a decode batch, and of a large prefill batch
        {"name": "quantize_16", "op": "quantize", "rows": 16, "K": 4096},
        {"name": "quantize_16384", "op": "quantize", "rows": 16384, "K": 4096},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "up", "down", "ffn", "select", "quantize"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "K": 32 * _log_int(rng, 2, 128)}
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * _log_int(rng, 4, 512 // groups)
        kept = rng.randint(1, groups)
        S = rng.randint(0, 1)
        c = _sel("", _log_int(rng, 1, 16384), E, S, rng.randint(1, min(10, kept * (E // groups))), rng.choice(["softmax", "sigmoid"]),
                 rng.random() < 0.7, groups, kept, rng.randint(1, 2), rng.choice(["fp32", "bf16"]), rng.random() < 0.7)
        del c["name"]
        return c
    while True:
        E = rng.choice([8, 16, 32, 60, 64, 128, 256, 512])
        case = {"op": op, "T": _log_int(rng, 1, 16384), "H": 32 * _log_int(rng, 8, 128), "E": E, "S": rng.randint(0, 1),
                "k": rng.randint(1, min(10, E)), "I": 32 * _log_int(rng, 4, 32), "A": rng.choice([64, 128]), "zipf": rng.choice([0.0, 1.1])}
        slots = case["T"] * (case["k"] + case["S"])
        if slots * case["H"] * case["I"] <= LARGE and (E + case["S"]) * case["H"] * case["I"] <= WEIGHTS and slots <= 131072:
            return case


# ------------------------------------------------------------------ inputs --


def _blocks(x, dims):
    """x padded with zeros to whole blocks of BLOCK along its last `dims` dimensions, those split in two."""
    pad = []
    for d in range(1, dims + 1):
        pad += [0, -x.shape[-d] % BLOCK]
    x = torch.nn.functional.pad(x, pad)
    if dims == 1:
        return x.unflatten(-1, (-1, BLOCK))
    return x.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))


def _scaled(x32, amax):
    """x over the scale amax / 448 (which is kept at 2^-110 / 448 or above), 0 in a block of zeros."""
    inv = torch.full_like(amax, 448.0) / amax.clamp(min=2.0 ** -110)  # (a quotient by or of a plain number is rounded twice)
    return torch.where(amax > 0, x32 * inv, torch.zeros_like(x32))


def _scale(amax):
    return torch.where(amax > 0, amax.clamp(min=2.0 ** -110) / torch.full_like(amax, 448.0), torch.zeros_like(amax))


def _quantize(x):
    """E4M3 codes (uint8, like x) of rows [..., K], and one fp32 scale per 128 values [..., ceil(K / 128)]."""
    b = _blocks(x.float(), 1)
    amax = b.abs().amax(-1, keepdim=True)
    q = _scaled(b, amax).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)[..., : x.shape[-1]]
    return q.contiguous(), _scale(amax).squeeze(-1)


def _quantize_weight(w):
    """The same of matrices [..., N, K], one scale per 128 x 128 block [..., ceil(N / 128), ceil(K / 128)]."""
    b = _blocks(w.float(), 2)
    amax = b.abs().amax((-1, -3), keepdim=True)
    q = _scaled(b, amax).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2).flatten(-3, -2)
    return q[..., : w.shape[-2], : w.shape[-1]].contiguous(), _scale(amax).squeeze(-1).squeeze(-2)


def _values(codes, scales):
    """fp32 values of rows of codes."""
    v = codes.view(torch.float8_e4m3fn).float()
    return v * scales.repeat_interleave(BLOCK, -1)[..., : v.shape[-1]]


def _weight_values(codes, scales):
    rows = scales.repeat_interleave(BLOCK, -2)[..., : codes.shape[-2], :]
    return _values(codes, rows)


def _route(case, gen):
    """Ids and weights as the router gives them, and the align's sorted slots, block owners and padded length."""
    T, E, S, k, A = case["T"], case["E"], case["S"], case["k"], case["A"]
    prior = -case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    noise = -torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=gen).clamp(1e-9, 1 - 1e-7)))
    top = (prior + noise).topk(k, dim=1)
    ids, wts = top.indices.int(), torch.softmax(top.values, 1)
    if S:
        ids = torch.cat([ids, torch.full((T, 1), E, dtype=torch.int32, device="cuda")], 1)
        wts = torch.cat([wts, torch.sigmoid(torch.randn(T, 1, device="cuda", generator=gen))], 1)
    width, Ea = k + S, E + S
    numel = T * width
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    count = torch.bincount(flat, minlength=Ea)
    padded = (count + A - 1) // A * A
    start = torch.cumsum(padded, 0) - padded
    first = torch.cumsum(count, 0) - count
    cap = numel + Ea * (A - 1)
    srt = torch.full((cap,), numel, dtype=torch.int32, device="cuda")
    place = start[flat[order]] + torch.arange(numel, device="cuda") - first[flat[order]]
    srt[place] = order.int()
    eids = torch.zeros((cap + A - 1) // A, dtype=torch.int32, device="cuda")
    owners = torch.repeat_interleave(torch.arange(Ea, device="cuda"), padded // A)
    eids[: owners.numel()] = owners.int()
    npp = padded.sum().int().view(1)
    return {"ids": ids.contiguous(), "wts": wts.float().contiguous(), "sorted": srt, "eids": eids, "npp": npp, "blocks": int(owners.numel())}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=dtype).mul_(std)

    def weight(matrices, N, K):  # quantised once, as a program that serves 8-bit experts keeps it
        # (16 matrices at a time: the intermediate values are in 32 bits)
        parts = [_quantize_weight(p) for p in normal(matrices, N, K, std=K ** -0.5).split(16)]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])

    if case["op"] == "quantize":
        return {"case": case, "x": normal(case["rows"], case["K"])}
    if case["op"] == "select":
        T, E = case["T"], case["E"]
        dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        # experts of different popularity; the balance bias leans against it
        lean = normal(E, std=0.5, dtype=torch.float32)
        logits = (normal(T, E, std=1.2, dtype=torch.float32) + lean).to(dtype)
        s = {"case": case, "logits": logits, "bias": None, "shared": None}
        if case["bias"]:
            s["bias"] = -0.1 * lean + normal(E, std=0.02, dtype=torch.float32)
        if case["S"]:
            s["shared"] = normal(T, dtype=torch.float32)
        return s
    T, H, I, Ea, width = case["T"], case["H"], case["I"], case["E"] + case["S"], case["k"] + case["S"]
    s = dict(_route(case, gen), case=case)
    if case["op"] != "down":  # the hidden states come as codes: the router's launch writes them
        s["x"], s["xs"] = _quantize(normal(T, H))
        w, ws = weight(2 * Ea, I, H)
        s["w13"], s["ws13"] = w.view(Ea, 2 * I, H), ws.view(Ea, -1, ws.shape[-1])
    else:
        g = normal(T * width, I)
        s["x"] = g * torch.sigmoid(g) * normal(T * width, I)
    if case["op"] != "up":
        s["w2"], s["ws2"] = weight(Ea, H, I)
    return s


# --------------------------------------------------------------------- run --


def _finite(x):
    """Logits in 64 bits, as far as they enter the scores: NaN and -inf as the lowest finite value, +inf as the largest."""
    big = torch.finfo(torch.float32).max
    return torch.nan_to_num(x.double(), nan=-big, posinf=big, neginf=-big)


def _select(logits, bias, shared, c):
    """Ids and weights; choices in 64 bits, as their order is what the ids are."""
    x = _finite(logits)
    T, E = x.shape
    if c["scoring"] == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        p = torch.exp(x - x.amax(1, keepdim=True))
        s = p / p.sum(1, keepdim=True)
    choice = s if bias is None else s + bias.double()
    G = c["groups"]
    if G > 1:
        best = torch.sort(choice.view(T, G, E // G), dim=-1, descending=True).values[..., : c["best"]].sum(-1)
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, : c["kept"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        stays[torch.arange(T, device=x.device)[:, None], kept] = True
        choice = torch.where(stays.repeat_interleave(E // G, 1), choice, torch.full_like(choice, -math.inf))
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, : c["k"]]
    w = torch.gather(s, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * 2.5
    if c["S"]:
        ids = torch.cat([ids, torch.full((T, 1), E, dtype=ids.dtype, device=ids.device)], 1)
        w = torch.cat([w, 1 / (1 + torch.exp(-shared.double()))[:, None]], 1)
    return ids.int(), w


def _plain_rows(s, which):
    """The blocks' slots [blocks, A], which of them are real, and the blocks' weights in 32 bits."""
    c, n = s["case"], s["blocks"]
    rows = s["sorted"][: n * c["A"]].view(n, c["A"]).long()
    real = rows < s["ids"].numel()
    e = s["eids"][:n]
    w, ws = s["w" + which][e], s["ws" + which][e]
    if which == "13":  # the gate's and the up rows' blocks apart
        w = _weight_values(w.unflatten(1, (2, -1)), ws.unflatten(1, (2, -1))).flatten(1, 2)
    else:
        w = _weight_values(w, ws)
    return rows, real, w


def _plain_up(s, x):
    c = s["case"]
    I, numel = c["I"], s["ids"].numel()
    rows, real, w = _plain_rows(s, "13")
    h = torch.bmm(x[torch.where(real, rows // (c["k"] + c["S"]), 0)], w.transpose(1, 2))
    g, u = h[..., :I], h[..., I:]
    act = g / (1 + torch.exp(-g)) * u
    out = torch.empty(numel + 1, I, dtype=torch.bfloat16, device=x.device)
    out[torch.where(real, rows, numel)] = act.to(torch.bfloat16)
    return out[:numel]


def _plain_down(s, x):
    c = s["case"]
    numel = s["ids"].numel()
    rows, real, w = _plain_rows(s, "2")
    y = torch.empty(numel + 1, c["H"], dtype=torch.float32, device=x.device)
    y[torch.where(real, rows, numel)] = torch.bmm(x[torch.where(real, rows, 0)], w.transpose(1, 2))
    return (y[:numel].view(c["T"], -1, c["H"]) * s["wts"][:, :, None]).sum(1).to(torch.bfloat16)


def _own(s):
    import moe_router_top_gb300 as smr

    c = s["case"]
    if c["op"] == "quantize":
        codes, scales = smr.quantize_fp8(s["x"])
        return smr.dequantize_fp8(codes, scales), scales
    if c["op"] == "select":
        return smr.select_experts(s["logits"], topk=c["k"], scoring=c["scoring"], balance_bias=s["bias"], num_groups=c["groups"],
                                  topk_groups=c["kept"], group_best=c["best"], renormalize=c["renorm"], routed_scale=2.5,
                                  has_shared=bool(c["S"]), shared_logits=s["shared"])
    al = (s["sorted"], s["eids"], s["npp"])
    if c["op"] == "down":
        x, xs = smr.quantize_fp8(s["x"])
    else:
        x = smr.expert_up(s["x"], s["w13"], *al, width=c["k"] + c["S"], block_size=c["A"], x_scales=s["xs"], w_scales=s["ws13"],
                          quantize_act=c["op"] == "ffn")
        if c["op"] == "up":
            return x
        x, xs = x
    return smr.expert_down(x, s["w2"], s["ids"], s["wts"], *al, block_size=c["A"], x_scales=xs, w_scales=s["ws2"])


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "select":
        ids, w = _select(state["logits"], state["bias"], state["shared"], c)
        return ids, w.float()
    if c["op"] == "quantize":
        codes, scales = _quantize(state["x"])
        return _values(codes, scales).to(torch.bfloat16), scales
    if c["op"] == "down":
        return _plain_down(state, _values(*_quantize(state["x"])))
    act = _plain_up(state, _values(state["x"], state["xs"]))
    return act if c["op"] == "up" else _plain_down(state, _values(*_quantize(act)))


# -------------------------------------------------------------------- work --


def _touched(case):
    """Expected number of experts with a row: an expert of share q is among a token's k with about
    1 - exp(-c q), c such that these sum to k; plus the shared one."""
    E, k = case["E"], case["k"]
    q = [(r + 1.0) ** -case["zipf"] for r in range(E)]
    tot = sum(q)
    lo, hi = 0.0, 1e9
    for _ in range(200):
        c = (lo + hi) / 2
        lo, hi = (c, hi) if sum(1 - math.exp(-c * v / tot) for v in q) < k else (lo, c)
    return sum(1 - math.exp(-lo * v / tot * case["T"]) for v in q) + case["S"]


def work(case):
    if case["op"] == "quantize":  # bf16 and bf16 values, and the scales (the codes between them are written too)
        n = case["rows"] * case["K"]
        return {"bytes": n * (2 + 1 + 2) + 4 * case["rows"] * math.ceil(case["K"] / BLOCK), "flops": 2 * n}
    if case["op"] == "select":
        n, out = case["T"] * case["E"], case["T"] * (case["k"] + case["S"])
        return {"bytes": n * (4 if case["dtype"] == "fp32" else 2) + 8 * out + 4 * case["E"] * case["bias"] + 4 * case["T"] * case["S"],
                "flops": 20 * n}
    T, H, I = case["T"], case["H"], case["I"]
    n = T * (case["k"] + case["S"])
    wide = {"up": 2, "down": 1, "ffn": 3}[case["op"]]
    byte = 1 + 4 / BLOCK  # of an activation
    acts = {"up": T * H * byte + 2 * n * I, "down": 2 * n * I + 2 * T * H, "ffn": T * H * byte + 2 * T * H}[case["op"]]
    return {"bytes": _touched(case) * wide * H * I * (1 + 4 / BLOCK ** 2) + acts + 8 * n, "flops": 2 * wide * n * H * I}


# ------------------------------------------------------------------- exact --


def _exact_e4m3(x):
    """What rows hold after quantisation, and the scales, from the definition: per 128 values the scale is
    amax / 448 and the factor 448 / amax, each a 32-bit number; a value's code is the E4M3 number nearest to its
    (32-bit) product with the factor, halves to the even one."""
    K = x.shape[-1]
    parts, scales = [], []
    for b in range(0, K, BLOCK):
        v = x[..., b : b + BLOCK].double()
        top = v.abs().amax(-1, keepdim=True)
        some = top > 0
        top = torch.where(some, top.clamp(min=2.0 ** -110), torch.ones_like(top))
        scale = torch.where(some, (top / 448).float().double(), torch.zeros_like(top))
        v = (v * (448 / top).float().double()).float().double()
        unit = torch.exp2(torch.frexp(v).exponent.double().clamp(min=-5) - 4)  # 8 to 16 units in a power of two; 2^-9 below 2^-6
        parts.append((torch.round(v / unit) * unit).clamp(-448, 448) * scale)
        scales.append(scale)
    return torch.cat(parts, -1), torch.cat(scales, -1)


def _exact_weight(codes, scales):
    """Codes' values: sign, 4 bits of exponent, 3 of mantissa (1 + m / 8) 2^(e - 7), e = 0: (m / 8) 2^-6."""
    c = codes.int()
    e, m = (c >> 3) & 15, (c & 7).double() / 8
    v = torch.where(e > 0, (1 + m) * torch.exp2(e.double() - 7), m * 2.0 ** -6) * (1 - 2 * (c >> 7).double())
    N, K = codes.shape
    n = torch.arange(N, device=codes.device) // BLOCK
    k = torch.arange(K, device=codes.device) // BLOCK
    return v * scales.double()[n][:, k]


def _exact_select(s):
    """From the definition, a greedy pick at a time: the largest choice that is left, the first of equal ones."""
    c, x = s["case"], s["logits"].double()
    T, E = x.shape
    score = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, 1)
    choice = score if s["bias"] is None else score + s["bias"].double()
    G, row = c["groups"], torch.arange(T, device=x.device)
    if G > 1:
        left = choice.reshape(T, G, E // G)
        total = left.topk(min(c["best"], E // G), dim=-1).values.sum(-1)
        masked = torch.full_like(left, -math.inf)
        for _ in range(c["kept"]):
            g = (total == total.amax(1, keepdim=True)).int().argmax(1)
            masked[row, g] = left[row, g]
            total[row, g] = -math.inf
        choice = masked.reshape(T, E)
    choice = choice.clone()
    ids = torch.empty(T, c["k"], dtype=torch.long, device=x.device)
    for j in range(c["k"]):
        ids[:, j] = (choice == choice.amax(1, keepdim=True)).int().argmax(1)
        choice[row, ids[:, j]] = -math.inf
    w = score[row[:, None], ids]
    w = 2.5 * (w / w.sum(1, keepdim=True) if c["renorm"] else w)
    if c["S"]:
        ids = torch.cat([ids, torch.full_like(ids[:, :1], E)], 1)
        w = torch.cat([w, torch.sigmoid(s["shared"].double())[:, None]], 1)
    return ids.int(), w


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_e4m3(s["x"])
    if case["op"] == "select":
        return _exact_select(s)
    I, ids, width = case["I"], s["ids"].reshape(-1), case["k"] + case["S"]
    slots = [(e, torch.nonzero(ids == e).squeeze(1)) for e in torch.unique(ids).tolist()]
    if case["op"] == "down":
        x = _exact_e4m3(s["x"])[0]
    else:
        x = _exact_weight_rows(s["x"], s["xs"])
        act = torch.zeros(ids.numel(), I, dtype=torch.float64, device="cuda")
        for e, i in slots:
            half = s["ws13"].shape[1] // 2
            g = x[i // width] @ _exact_weight(s["w13"][e, :I], s["ws13"][e, :half]).T
            u = x[i // width] @ _exact_weight(s["w13"][e, I:], s["ws13"][e, half:]).T
            act[i] = g * torch.sigmoid(g) * u
        if case["op"] == "up":
            return act
        x = _exact_e4m3(act.to(torch.bfloat16))[0]  # quantised from the activations as bf16 holds them
    y = torch.zeros(ids.numel(), case["H"], dtype=torch.float64, device="cuda")
    for e, i in slots:
        y[i] = x[i] @ _exact_weight(s["w2"][e], s["ws2"][e]).T
    return (y.view(case["T"], width, -1) * s["wts"].double()[:, :, None]).sum(1)


def _exact_weight_rows(codes, scales):
    """Rows' values: a row is a matrix of one row for its scales."""
    k = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    ones = torch.ones(1, scales.shape[1], dtype=torch.float64, device=codes.device)
    parts = [_exact_weight(p, ones.expand((p.shape[0] + BLOCK - 1) // BLOCK, -1)) for p in codes.split(4096)]
    return torch.cat(parts) * scales.double()[:, k]
