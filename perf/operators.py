"""The experts' feed-forward behind the router: its cases, plain forms and exact values.

Operators: the grouped gated product (expert_up), the grouped product with the
weighted sum over a token's slots (expert_down), both with bf16 or MXFP4 weights
(the activations then quantised in the same pass), and MXFP4 quantisation with
its inverse. A routed slot i = t * width + s; w13 holds every expert's I gate
rows, then its I up rows.
"""
import math

import torch

own = False

LARGE = 16384 * 8 * 2048 * 768          # slots x H x I of the largest case
WEIGHTS = 513 * 512 * 4096              # experts x H x I of the largest weights


def _ffn(name, op, fmt, T, H, E, S, k, I, A, zipf=0.0):
    return {"name": name, "op": op, "fmt": fmt, "T": T, "H": H, "E": E, "S": S, "k": k, "I": I, "A": A, "zipf": zipf}


def listed():
    return [
        # speculative verify step, 512 experts and the shared one: latency, weights streamed
        _ffn("up_verify_4", "up", "bf16", 4, 4096, 512, 1, 10, 512, 64),
        # short prompt with a few hot experts: most experts hold a handful of rows
        _ffn("up_skewed_512", "up", "bf16", 512, 2048, 128, 0, 8, 768, 64, 1.1),
        # large prefill batch: about 1024 rows an expert
        _ffn("up_large_16384", "up", "bf16", 16384, 2048, 128, 0, 8, 768, 128),
        # one sequence decoding one token: the smallest call
        _ffn("down_token_1", "down", "bf16", 1, 2048, 128, 0, 8, 768, 64),
        # odd-sized prompt, skewed: ragged segments
        _ffn("down_skewed_2047", "down", "bf16", 2047, 2048, 128, 0, 8, 768, 128, 1.1),
        _ffn("down_large_16384", "down", "bf16", 16384, 2048, 128, 0, 8, 768, 128),
        # 4-bit experts: a small decode batch, a ragged prompt, a large batch
        _ffn("up_mx_decode_8", "up", "mxfp4", 8, 4096, 512, 1, 10, 512, 64),
        _ffn("up_mx_large_16384", "up", "mxfp4", 16384, 2048, 128, 0, 8, 768, 128),
        _ffn("down_mx_decode_8", "down", "mxfp4", 8, 4096, 512, 1, 10, 512, 64),
        _ffn("down_mx_ragged_1021", "down", "mxfp4", 1021, 2048, 128, 0, 8, 768, 64, 1.1),
        # hidden states of a decode batch, and of a large prefill batch
        {"name": "quantize_16", "op": "quantize", "rows": 16, "K": 4096},
        {"name": "quantize_16384", "op": "quantize", "rows": 16384, "K": 4096},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["up", "down", "up", "down", "quantize"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "K": 32 * _log_int(rng, 2, 128)}
    fmt = rng.choice(["bf16", "mxfp4"])
    step = 16 if fmt == "bf16" else 128
    while True:
        E = rng.choice([8, 16, 32, 60, 64, 128, 256, 512])
        case = {"op": op, "fmt": fmt, "T": _log_int(rng, 1, 16384), "H": step * max(1, _log_int(rng, 256, 4096) // step), "E": E,
                "S": rng.randint(0, 1), "k": rng.randint(1, min(10, E)), "I": step * max(1, _log_int(rng, 128, 1024) // step),
                "A": rng.choice([64, 128]), "zipf": rng.choice([0.0, 1.1])}
        slots = case["T"] * (case["k"] + case["S"])
        if slots * case["H"] * case["I"] <= LARGE and (E + case["S"]) * case["H"] * case["I"] <= WEIGHTS and slots <= 131072:
            return case


# ------------------------------------------------------------------ inputs --


def _e2m1_round(v):
    """The code (0..7) of the E2M1 value nearest to v >= 0, ties to the even code, saturated at 6."""
    code = (v > 0.25).to(torch.uint8)
    code += v >= 0.75
    code += v > 1.25
    code += v >= 1.75
    code += v > 2.5
    code += v >= 3.5
    code += v > 5.0
    return code


def _mx_scale_exp(x32):
    """Exponent e of the blocks' scale 2^e: the smallest power of two with amax / 2^e <= 6, e >= -127."""
    amax = x32.abs().amax(-1, keepdim=True)
    m, p = torch.frexp(amax)  # amax = m 2^p, m in [0.5, 1): 6 * 2^e = 0.75 * 2^(e + 3)
    e = torch.where(m > 0.75, p - 2, p - 3)
    return torch.where(amax > 0, e.clamp(min=-127), torch.full_like(e, -127))


def _mx_pow2(e):
    """2^e as float32, e in [-127, 127], in two factors (2^-127 is below the smallest normal number)."""
    h = torch.div(e, 2, rounding_mode="floor")
    return torch.ldexp(torch.ones_like(h, dtype=torch.float32), h), torch.ldexp(torch.ones_like(h, dtype=torch.float32), e - h)


def _mx_quantize(x):
    """MXFP4 codes (uint8 [..., K / 2], the even element in the low half) and E8M0 scale bytes [..., K / 32]."""
    b = x.float().unflatten(-1, (-1, 32))
    e = _mx_scale_exp(b)
    s0, s1 = _mx_pow2(-e)
    v = b * s0 * s1
    code = (_e2m1_round(v.abs()) + 8 * torch.signbit(b)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (e.squeeze(-1) + 127).to(torch.uint8)


def _mx_values(codes, scales):
    """float32 values of codes [..., K / 2] and scale bytes [..., K / 32]."""
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    grid += [-g for g in grid]
    pairs = torch.tensor([[grid[c & 15], grid[c >> 4]] for c in range(256)], dtype=torch.float32, device=codes.device)
    v = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    s0, s1 = _mx_pow2(scales.int() - 127)
    return (v * s0.unsqueeze(-1) * s1.unsqueeze(-1)).flatten(-2)


def _tile_scales(scales, gated):
    """Row-major scales [E, N, K / 32] in the order that the products read: 128-row tiles of 512-byte
    pieces of 4 blocks. gated: a tile holds 64 features, 16 gate rows and their 16 up rows in turn."""
    E, N, B = scales.shape
    if gated:
        t = torch.nn.functional.pad(scales.view(E, 2, N // 2, B), (0, 0, 0, -(N // 2) % 64))
        return t.view(E, 2, -1, 4, 16, B // 4, 4).permute(0, 2, 5, 1, 4, 3, 6).reshape(E, -1, B // 4, 512).contiguous()
    t = torch.nn.functional.pad(scales, (0, 0, 0, -N % 128))
    return t.view(E, -1, 4, 32, B // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, -1, B // 4, 512).contiguous()


def _untile_scales(tiled, N, gated):
    n, t, c, _ = tiled.shape
    if gated:
        return tiled.view(n, t, c, 2, 16, 4, 4).permute(0, 3, 1, 5, 4, 2, 6).reshape(n, 2, t * 64, c * 4)[:, :, : N // 2].reshape(n, N, c * 4)
    return tiled.view(n, t, c, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, t * 128, c * 4)[:, :N]


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

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=torch.bfloat16).mul_(std)

    if case["op"] == "quantize":
        return {"case": case, "x": normal(case["rows"], case["K"])}
    T, H, I, Ea, width = case["T"], case["H"], case["I"], case["E"] + case["S"], case["k"] + case["S"]
    s = dict(_route(case, gen), case=case)
    if case["op"] == "up":
        s["x"] = normal(T, H)
        w = normal(Ea, 2 * I, H, std=H ** -0.5)
    else:
        g = normal(T * width, I)
        s["x"] = g * torch.sigmoid(g) * normal(T * width, I)
        w = normal(Ea, H, I, std=I ** -0.5)
    if case["fmt"] == "bf16":
        s["w"] = w
    else:  # laid out once, as a program that serves 4-bit experts keeps them
        # (16 experts at a time: the intermediate values are in 32 bits)
        parts = [_mx_quantize(p) for p in w.split(16)]
        s["w"] = torch.cat([p[0] for p in parts]).to(torch.uint8)
        s["w_scales"] = _tile_scales(torch.cat([p[1] for p in parts]), case["op"] == "up")
    return s


# --------------------------------------------------------------------- run --


def _plain_rows(s):
    """The blocks' slots [blocks, A], which of them are real, and the blocks' weights in 32 bits."""
    c, n = s["case"], s["blocks"]
    rows = s["sorted"][: n * c["A"]].view(n, c["A"]).long()
    real = rows < s["ids"].numel()
    e = s["eids"][:n]
    if c["fmt"] == "bf16":
        w = s["w"][e].float()
    else:
        up = c["op"] == "up"
        w = _mx_values(s["w"][e], _untile_scales(s["w_scales"][e], 2 * c["I"] if up else c["H"], up))
    return rows, real, w


def _plain_x(s):
    return s["x"].float() if s["case"]["fmt"] == "bf16" else _mx_values(*_mx_quantize(s["x"]))


def _plain_up(s):
    c = s["case"]
    I, numel = c["I"], s["ids"].numel()
    rows, real, w = _plain_rows(s)
    x = _plain_x(s)[torch.where(real, rows // (c["k"] + c["S"]), 0)]
    h = torch.bmm(x, w.transpose(1, 2))
    g, u = h[..., :I], h[..., I:]
    act = g / (1 + torch.exp(-g)) * u
    out = torch.empty(numel + 1, I, dtype=torch.bfloat16, device=x.device)
    out[torch.where(real, rows, numel)] = act.to(torch.bfloat16)
    return out[:numel]


def _plain_down(s):
    c = s["case"]
    numel = s["ids"].numel()
    rows, real, w = _plain_rows(s)
    x = _plain_x(s)[torch.where(real, rows, 0)]
    y = torch.empty(numel + 1, c["H"], dtype=torch.float32, device=x.device)
    y[torch.where(real, rows, numel)] = torch.bmm(x, w.transpose(1, 2))
    return (y[:numel].view(c["T"], -1, c["H"]) * s["wts"][:, :, None]).sum(1).to(torch.bfloat16)


def _own(s):
    import moe_router_top_gb300 as smr

    c = s["case"]
    if c["op"] == "quantize":
        return smr.dequantize_mxfp4(*smr.quantize_mxfp4(s["x"]))
    x, scales = s["x"], {}
    if c["fmt"] == "mxfp4":
        x, xs = smr.quantize_mxfp4(x)
        scales = {"x_scales": xs, "w_scales": s["w_scales"]}
    if c["op"] == "up":
        return smr.expert_up(x, s["w"], s["sorted"], s["eids"], s["npp"], width=c["k"] + c["S"], block_size=c["A"], **scales)
    return smr.expert_down(x, s["w"], s["ids"], s["wts"], s["sorted"], s["eids"], s["npp"], block_size=c["A"], **scales)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "quantize":
        return _mx_values(*_mx_quantize(state["x"])).to(torch.bfloat16)
    return _plain_up(state) if op == "up" else _plain_down(state)


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
    if case["op"] == "quantize":  # bf16 in, bf16 values out (the codes and scales between them are written too)
        n = case["rows"] * case["K"]
        return {"bytes": n * (2 + 17 / 32 + 2), "flops": 2 * n}
    T, H, I = case["T"], case["H"], case["I"]
    n = T * (case["k"] + case["S"])
    per = 2 if case["fmt"] == "bf16" else 17 / 32
    wide = 2 if case["op"] == "up" else 1
    weights = _touched(case) * wide * H * I * per
    acts = 2 * (T * H + n * I)
    return {"bytes": weights + acts + 8 * n, "flops": 2 * wide * n * H * I}


# ------------------------------------------------------------------- exact --


def _exact_mx(x):
    """x as MXFP4 holds it, in 64 bits: each 32 values over 2^ceil(log2(amax / 6)), to the nearest
    multiple of 1/2 (below 2), 1 (below 4) or 2, halves to the even one."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    m, p = torch.frexp(top / 6)
    e = torch.where(m == 0.5, p - 1, p).clamp(min=-127)
    s = torch.where(top > 0, torch.exp2(e.double()), torch.ones_like(top))
    v = b / s
    unit = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    return ((torch.round(v / unit) * unit) * s).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_mx(s["x"])
    up, mx = case["op"] == "up", case["fmt"] == "mxfp4"
    x = _exact_mx(s["x"]) if mx else s["x"].double()
    ids, width = s["ids"].reshape(-1), case["k"] + case["S"]
    out = torch.zeros(ids.numel(), case["I"] if up else case["H"], dtype=torch.float64, device="cuda")
    for e in torch.unique(ids).tolist():
        w = s["w"][e]
        if mx:  # nibbles to values: (-1)^s * (m / 2) for exponent 0, (1 + m / 2) * 2^(exponent - 1) else
            nib = torch.stack([w & 15, w >> 4], -1).flatten(-2).double()
            sign = 1 - 2 * (nib >= 8).double()
            mag = nib % 8
            ex, m = torch.floor(mag / 2), mag % 2
            val = sign * torch.where(ex > 0, (1 + m / 2) * torch.exp2(ex - 1), m / 2)
            sc = _untile_scales(s["w_scales"][e : e + 1], w.shape[0], up)[0]
            w = (val.unflatten(-1, (-1, 32)) * torch.exp2(sc.double() - 127).unsqueeze(-1)).flatten(-2)
        else:
            w = w.double()
        i = torch.nonzero(ids == e).squeeze(1)
        h = x[i // width if up else i] @ w.T
        if up:
            g, u = h[:, : case["I"]], h[:, case["I"] :]
            h = g * torch.sigmoid(g) * u
        out[i] = h
    if up:
        return out
    return (out.view(case["T"], width, -1) * s["wts"].double()[:, :, None]).sum(1)
