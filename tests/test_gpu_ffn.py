"""The experts' feed-forward (gated product, weighted second product) in bf16
and MXFP4, and MXFP4 quantisation, against plain 64-bit forms. Needs a GB300.

Bounds (u = 2^-8, half a bf16 step; c = 2 (K/16 + 32) 2^-24, fp32 accumulation
in the tensor core, one update per 16 values of K, of a sum of magnitudes ad):
  up:   |da| <= 1.1 |u| c ad_g + |silu(g)| c ad_u + (8 + 1.2 |g|) 2^-23 |a| + u |a|
        (|silu'| <= 1.1; the fast exponential is off by 2 + 1.2 |g| units of
        2^-23, the division, sum and product by a few more; the cross term of
        both errors is inside the factor 2 of c), and half the smallest
        subnormal bf16, 2^-134
  down: |do| <= sum_s |w_s| (c ad_s + u |y_s|) (1 + u) + width 2^-24 sum_s |w_s y_s| + u |o| + 2^-134
"""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def smr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import moe_router_top_gb300 as m
    return m


U = 2.0 ** -8
TINY = 2.0 ** -134


def _routing(T, E, k, S, zipf, seed):
    """Ids (k distinct experts a token, then the shared one) and weights."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    prior = -zipf * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float64))
    z = prior - torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=g, dtype=torch.float64).clamp(1e-12)))
    ids = z.topk(k, 1).indices.int()
    wts = torch.rand(T, k + S, device="cuda", generator=g)
    if S:
        ids = torch.cat([ids, torch.full((T, 1), E, dtype=torch.int32, device="cuda")], 1)
    return ids.contiguous(), wts, g


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(torch.bfloat16)


GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _mx_exact(x):
    """(codes, scale bytes, values) of x in 64 bits: the definition, by comparing distances to the grid."""
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    m, p = torch.frexp(amax / 6)
    e = torch.where(m == 0.5, p - 1, p).clamp(min=-127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    v = b / torch.exp2(e.double())
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    d = (v.abs().unsqueeze(-1) - grid).abs()
    best = d.amin(-1, keepdim=True)
    near = d == best  # one or two neighbours: of two, the even code
    idx = torch.arange(8, device=x.device)
    code = torch.where(near & (idx % 2 == 0), idx, -1).amax(-1)
    code = torch.where(near.sum(-1) == 1, near.int().argmax(-1), code)
    val = grid[code] * torch.where(v < 0, -1.0, 1.0) * torch.exp2(e.double())
    code = (code + 8 * torch.signbit(b)).flatten(-2)
    packed = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
    return packed, (e.squeeze(-1) + 127).to(torch.uint8), val.flatten(-2)


def _ref_up(x, w, ids, width):
    """act and its error bound, float64 (x [T, H], w [E, 2I, H])."""
    K, I = x.shape[1], w.shape[1] // 2
    c = 2.0 * (K // 16 + 32) * 2.0 ** -24
    out = torch.zeros(ids.numel(), I, dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(out)
    flat = ids.reshape(-1)
    for e in torch.unique(flat).tolist():
        if e < 0 or e >= w.shape[0]:
            continue
        i = torch.nonzero(flat == e).squeeze(1)
        h, ad = x[i // width] @ w[e].T, x[i // width].abs() @ w[e].abs().T
        g, u, ag, au = h[:, :I], h[:, I:], ad[:, :I], ad[:, I:]
        s = g / (1 + torch.exp(-g))
        a = s * u
        out[i] = a
        tol[i] = (1.1 * u.abs() * c * ag + s.abs() * c * au + (8 + 1.2 * g.abs()) * 2.0 ** -23 * a.abs()) * (1 + U) + U * a.abs() + TINY
    return out, tol


def _ref_down(x, w, ids, wts):
    T, width = ids.shape
    K, H = x.shape[1], w.shape[1]
    c = 2.0 * (K // 16 + 32) * 2.0 ** -24
    y = torch.zeros(ids.numel(), H, dtype=torch.float64, device=x.device)
    dy = torch.zeros_like(y)
    flat = ids.reshape(-1)
    for e in torch.unique(flat).tolist():
        if e < 0 or e >= w.shape[0]:
            continue
        i = torch.nonzero(flat == e).squeeze(1)
        y[i] = x[i] @ w[e].T
        dy[i] = c * (x[i].abs() @ w[e].abs().T)
    dy = dy * (1 + U) + U * y.abs() + TINY
    wt = wts.double()[:, :, None]
    y, dy = y.view(T, width, H), dy.view(T, width, H)
    out = (wt * y).sum(1)
    mag = (wt.abs() * y.abs()).sum(1)
    tol = (wt.abs() * dy).sum(1) * (1 + U) + width * 2.0 ** -24 * mag + U * out.abs() + TINY
    return out, tol


def _close(got, ref, tol):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), "not every routed row was written"
    assert (err <= tol).all(), f"max error / bound {(err / tol).max().item():.3g}"


def _laid_out(smr, w, gated, **kw):
    codes, scales = smr.quantize_mxfp4(w, **kw)
    return codes, smr.tile_mxfp4_scales(scales, gated=gated, **kw)


def _weights_mx(smr, w, gated):
    return *_laid_out(smr, w, gated), _mx_exact(w)[2]


def _values(smr, x, mx):
    """What a product is called with, and the 64-bit values that it stands for."""
    if not mx:
        return x, {}, x.double()
    codes, scales = smr.quantize_mxfp4(x)
    return codes, {"x_scales": scales}, _mx_exact(x)[2]


# T, H, I, E, S, k, A, zipf
SHAPES = [
    (1, 16, 16, 1, 0, 1, 64, 0.0),        # one of everything
    (1, 2048, 768, 128, 0, 8, 64, 0.0),   # a single token
    (3, 80, 48, 5, 1, 2, 64, 0.0),        # odd sizes, partial tiles and k-blocks
    (16, 256, 64, 4, 0, 4, 128, 0.0),     # 16 rows: whole columns
    (17, 272, 144, 7, 0, 3, 128, 0.0),    # one row more than 16
    (65, 144, 176, 3, 1, 2, 64, 0.0),     # a second block of one row
    (300, 512, 192, 64, 1, 8, 64, 1.1),
    (1000, 256, 128, 16, 0, 4, 128, 2.0),  # hot experts over many blocks
    (2500, 128, 80, 6, 1, 3, 64, 0.0),
    (4000, 400, 208, 5, 0, 2, 128, 0.0),  # pairs of CTAs: whole and partial tiles and k-blocks
    (3000, 272, 336, 4, 1, 1, 64, 1.1),   # pairs, an odd number of weight tiles, groups of four blocks
]
SHAPES_MX = [
    (1, 128, 128, 1, 0, 1, 64, 0.0),
    (1, 2048, 768, 128, 0, 8, 64, 0.0),
    (5, 384, 384, 6, 1, 2, 64, 0.0),      # K % 256 = 128: half a k-block
    (40, 256, 128, 3, 0, 2, 128, 0.0),
    (300, 512, 256, 64, 1, 8, 64, 1.1),
    (1000, 256, 640, 16, 0, 4, 128, 2.0),
    (2000, 384, 384, 5, 1, 2, 64, 0.0),   # pairs of CTAs, half a k-block
    (1500, 640, 256, 4, 0, 2, 128, 1.1),
]
# output features in partial tiles (only the contraction is in whole scale groups)
UP_MX = SHAPES_MX + [(20, 256, 80, 3, 0, 2, 64, 0.0), (600, 256, 208, 3, 0, 2, 64, 0.0), (700, 128, 176, 4, 1, 1, 128, 0.0)]
DOWN_MX = SHAPES_MX + [(20, 80, 256, 3, 0, 2, 64, 0.0), (600, 272, 256, 3, 0, 2, 64, 0.0), (700, 400, 128, 4, 1, 1, 128, 0.0)]


@pytest.mark.parametrize("mx,shape", [(False, s) for s in SHAPES] + [(True, s) for s in UP_MX])
def test_up_matches_64_bits(smr, mx, shape):
    T, H, I, E, S, k, A, zipf = shape
    ids, _, g = _routing(T, E, k, S, zipf, 11 + T)
    srt, eids, npp = smr.align(ids, E + S, A)
    x, w = _normal(g, T, H), _normal(g, E + S, 2 * I, H, std=1.5 * H ** -0.5)
    xa, kw, xv = _values(smr, x, mx)
    if mx:
        w, kw["w_scales"], wv = _weights_mx(smr, w, True)
    else:
        wv = w.double()
    out = torch.full((T * (k + S), I), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = smr.Workspace()
    smr.expert_up(xa, w, srt, eids, npp, width=k + S, block_size=A, out=out, workspace=ws, **kw)
    assert smr.get_device_error(ws) == 0 and smr.last_launch_count() == 1
    _close(out, *_ref_up(xv, wv, ids, k + S))


@pytest.mark.parametrize("mx,shape", [(False, s) for s in SHAPES] + [(True, s) for s in DOWN_MX])
def test_down_matches_64_bits(smr, mx, shape):
    T, H, I, E, S, k, A, zipf = shape
    ids, wts, g = _routing(T, E, k, S, zipf, 31 + T)
    srt, eids, npp = smr.align(ids, E + S, A)
    x, w = _normal(g, T * (k + S), I), _normal(g, E + S, H, I, std=I ** -0.5)
    xa, kw, xv = _values(smr, x, mx)
    if mx:
        w, kw["w_scales"], wv = _weights_mx(smr, w, False)
    else:
        wv = w.double()
    ws = smr.Workspace()
    out = smr.expert_down(xa, w, ids, wts, srt, eids, npp, block_size=A, workspace=ws, **kw)
    assert smr.get_device_error(ws) == 0
    _close(out, *_ref_down(xv, wv, ids, wts))


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 2048), (257, 4096), (1000, 160)])
def test_quantize_is_the_definition(smr, rows, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + K)
    x = _normal(g, rows, K) * torch.exp2(torch.randint(-120, 120, (rows, 1), generator=g, device="cuda").float())
    x = x.to(torch.bfloat16)
    # every magnitude border: multiples of 1/4 times powers of two, zeros, the
    # smallest and largest values of bf16
    x[0, :32] = torch.arange(32, device="cuda") * 0.25 - 4.0
    if rows > 2:
        x[1] = 0.0
        x[1, 5] = -0.0
        x[2, :32] = torch.tensor([6.0, -6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, 4.5, 0.26] + [0.0] * 20)
        x[2, 32:64] = 2.0 ** -133
        x[2, 64:96] = 3.3895313892515355e38
        x[2, 70] = -1.0
    codes, scales = smr.quantize_mxfp4(x)
    rc, rs, rv = _mx_exact(x)
    assert torch.equal(scales, rs)
    assert torch.equal(codes, rc)
    # exact in bf16, but for the largest bf16 values: 1.99 * 2^127 / 2^126 rounds to the
    # code 4, and 4 * 2^126 = 2^128 is above bf16's largest finite value, so it is infinite
    back = smr.dequantize_mxfp4(codes, scales)
    assert torch.equal(back.double(), torch.where(rv.abs() >= 2.0 ** 128, rv * float("inf"), rv))


def test_quantize_strided_and_special_blocks(smr):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    wide = _normal(g, 33, 256)
    part = wide[:, 64:192]
    codes, scales = smr.quantize_mxfp4(part)
    again = smr.quantize_mxfp4(part.contiguous())
    assert torch.equal(codes, again[0]) and torch.equal(scales, again[1])
    x = _normal(g, 2, 96)
    x[0, 3] = float("nan")
    x[1, 64] = float("-inf")
    codes, scales = smr.quantize_mxfp4(x)
    assert scales.tolist()[0][0] == 255 and scales.tolist()[1][2] == 255
    v = smr.dequantize_mxfp4(codes, scales)
    bad = torch.zeros(2, 96, dtype=torch.bool, device="cuda")
    bad[0, :32] = True
    bad[1, 64:] = True
    assert torch.equal(torch.isnan(v), bad)
    assert smr.quantize_mxfp4(x[:0])[0].shape == (0, 48)


def test_dequantize_every_code_and_scale(smr):
    codes = torch.arange(256, device="cuda").to(torch.uint8).repeat(256, 1)
    scales = torch.arange(256, device="cuda").to(torch.uint8)[:, None].repeat(1, 16)
    v = smr.dequantize_mxfp4(codes, scales)
    lut = torch.tensor(GRID + [-x for x in GRID], dtype=torch.float64, device="cuda")
    c = codes.long()
    ref = torch.stack([lut[c & 15], lut[c >> 4]], -1).flatten(-2) * torch.exp2(scales[:, :1].double() - 127)
    assert torch.isnan(v[255]).all()
    assert torch.equal(v[:255].double(), ref[:255].to(torch.bfloat16).double())


@pytest.mark.parametrize("E,N,K,gated", [(3, 160, 256, False), (2, 96, 384, True), (1, 32, 128, True), (5, 1, 128, False)])
def test_tiled_scales_layout(smr, E, N, K, gated):
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    s = torch.randint(0, 256, (E, N, K // 32), generator=g, device="cuda").to(torch.uint8)
    t = smr.tile_mxfp4_scales(s, gated=gated).cpu()
    s = s.cpu()
    I = N // 2
    for tile in range(t.shape[1]):
        for r in range(128):
            if gated:
                f = tile * 64 + (r // 32) * 16 + r % 16
                row = (r // 16 % 2) * I + f if f < I else None
            else:
                row = tile * 128 + r if tile * 128 + r < N else None
            for q in range(K // 32):
                got = t[:, tile, q // 4, (r % 32) * 16 + (r // 32) * 4 + q % 4]
                assert torch.equal(got, s[:, row, q] if row is not None else torch.zeros(E, dtype=torch.uint8))


def _case(smr, T=37, H=256, I=128, E=6, S=1, k=2, A=64, seed=3, mx=False):
    ids, wts, g = _routing(T, E, k, S, 0.0, seed)
    al = smr.align(ids, E + S, A)
    x, w13, w2 = _normal(g, T, H), _normal(g, E + S, 2 * I, H, std=1.5 * H ** -0.5), _normal(g, E + S, H, I, std=I ** -0.5)
    return ids, wts, al, x, w13, w2


def _ffn(smr, c, mx=False, **kw):
    ids, wts, al, x, w13, w2 = c
    ku, kd = {}, {}
    s = {"stream": kw["stream"]} if "stream" in kw else {}
    if mx:
        x, ku["x_scales"] = smr.quantize_mxfp4(x, **s)
        w13, ku["w_scales"] = _laid_out(smr, w13, True, **s)
    act = smr.expert_up(x, w13, *al, width=ids.shape[1], block_size=64, **ku, **kw)
    y = act
    if mx:
        y, kd["x_scales"] = smr.quantize_mxfp4(act, **s)
        w2, kd["w_scales"] = _laid_out(smr, w2, False, **s)
    return act, smr.expert_down(y, w2, ids, wts, *al, block_size=64, **kd, **kw)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,E,k,S", [(4, 64, 4, 1), (200, 32, 4, 0), (600, 4, 2, 1)])
def test_route_then_experts(smr, mx, T, E, k, S):
    """The whole layer as it is used: route and align, the gated product, the
    second product, each stage against 64 bits on the stage before it."""
    H, I = 512, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(T + E)
    x, gate = _normal(g, T, H), _normal(g, E, H, std=0.05)
    shared = _normal(g, 1, H, std=0.05) if S else None
    w13, w2 = _normal(g, E + S, 2 * I, H, std=H ** -0.5), _normal(g, E + S, H, I, std=I ** -0.5)
    ids, wts, *al = smr.route_align(x, gate, shared, topk=k, block_size=64)
    xa, kw, xv = _values(smr, x, mx)
    wa, wv = w13, w13.double()
    if mx:
        wa, kw["w_scales"], wv = _weights_mx(smr, w13, True)
    act = smr.expert_up(xa, wa, *al, width=k + S, block_size=64, **kw)
    _close(act, *_ref_up(xv, wv, ids, k + S))
    ya, kw, yv = _values(smr, act, mx)
    wa, wv = w2, w2.double()
    if mx:
        wa, kw["w_scales"], wv = _weights_mx(smr, w2, False)
    out = smr.expert_down(ya, wa, ids, wts, *al, block_size=64, **kw)
    _close(out, *_ref_down(yv, wv, ids, wts))


def test_strided_rows(smr):
    ids, wts, al, x, w13, w2 = _case(smr)
    wide = torch.full((x.shape[0], x.shape[1] + 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + x.shape[1]] = x
    part = wide[:, 8:8 + x.shape[1]]
    a = smr.expert_up(part, w13, *al, width=ids.shape[1], block_size=64)
    assert torch.equal(a, smr.expert_up(x, w13, *al, width=ids.shape[1], block_size=64))
    one = smr.expert_up(part[:1], w13, *smr.align(ids[:1].contiguous(), 7, 64), width=ids.shape[1], block_size=64)
    assert torch.equal(one, a[: ids.shape[1]])


def test_skipped_slots(smr):
    """Ids that no expert has (another rank's, say): their rows of act stay as
    they were and they add nothing, also where a whole token has none."""
    ids, wts, al, x, w13, w2 = _case(smr, T=50)
    ids = ids.clone()
    ids[3, 1], ids[7, 0], ids[20] = -1, 100, 7
    ws = smr.Workspace(256)
    al = smr.align(ids, 7, 64, workspace=ws)
    assert smr.get_device_error(ws) == 1
    out = torch.full((150, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    smr.expert_up(x, w13, *al, width=3, block_size=64, out=out)
    gone = ((ids < 0) | (ids >= 7)).reshape(-1)
    assert (out[gone] == 5.0).all() and gone.sum() == 5
    ref, tol = _ref_up(x.double(), w13.double(), ids, 3)
    _close(out[~gone], ref[~gone], tol[~gone])
    out[gone] = float("nan")
    y = smr.expert_down(out, w2, ids, wts, *al, block_size=64)
    clean = torch.where(gone[:, None], torch.zeros_like(out), out)
    _close(y, *_ref_down(clean.double(), w2.double(), ids, wts))
    assert (y[20] == 0).all()


def test_no_slot_at_all(smr):
    ids, wts, al, x, w13, w2 = _case(smr, T=5)
    ids = torch.full_like(ids, -1)
    al = smr.align(ids, 7, 64, workspace=smr.Workspace(256))
    assert int(al[2]) == 0
    act = torch.full((15, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    smr.expert_up(x, w13, *al, width=3, block_size=64, out=act)
    assert (act == 2.0).all()
    assert (smr.expert_down(act, w2, ids, wts, *al, block_size=64) == 0).all()


def test_remapped_experts(smr):
    """Behind an EPLB remap: the weights are the physical experts', the ids the logical ones'."""
    ids, wts, _, x, w13, w2 = _case(smr, T=90, E=6, S=0)
    phys = torch.tensor([[0, 7], [1, 1], [2, 8], [3, 3], [4, 4], [5, 6]], dtype=torch.int32, device="cuda")
    count = torch.tensor([2, 1, 2, 1, 1, 2], dtype=torch.int32, device="cuda")
    al = smr.align(ids, 6, 64, eplb_map=phys, eplb_count=count, num_physical=9)
    logical = torch.tensor([0, 1, 2, 3, 4, 5, 5, 0, 2], device="cuda")
    act = smr.expert_up(x, w13[logical].contiguous(), *al, width=2, block_size=64)
    _close(act, *_ref_up(x.double(), w13.double(), ids, 2))
    out = smr.expert_down(act, w2[logical].contiguous(), ids, wts, *al, block_size=64, num_logical=6)
    _close(out, *_ref_down(act.double(), w2.double(), ids, wts))


@pytest.mark.parametrize("mx", [False, True])
def test_captured_and_replayed(smr, mx):
    """Two graphs captured without a workspace of their own, replayed on two
    streams at once with new inputs between replays, next to eager calls."""
    cases = [_case(smr, T=40, seed=s) for s in (5, 6)]
    eager = [_ffn(smr, c, mx) for c in cases]
    graphs, outs = [], []
    for c in cases:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_ffn(smr, c, mx))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                gr.replay()
        again = _ffn(smr, cases[0], mx)
        assert torch.equal(again[1], eager[0][1])
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
    for got, ref in zip(outs, eager):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    cases[0][3].neg_()  # the first graph's hidden states
    graphs[0].replay()
    ref = _ffn(smr, cases[0], mx)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], ref[0]) and torch.equal(outs[0][1], ref[1])
    assert not torch.equal(ref[0], eager[0][0])


@pytest.mark.parametrize("mx", [False, True])
def test_streams(smr, mx):
    c = _case(smr, T=300)
    ref = _ffn(smr, c, mx)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [_ffn(smr, c, mx, stream=s) for s in streams for _ in range(4)]
    outs.append(_ffn(smr, c, mx, stream=streams[0].cuda_stream))
    with torch.cuda.stream(streams[1]):
        outs.append(_ffn(smr, c, mx))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], ref[0]) and torch.equal(o[1], ref[1])


def test_one_workspace_for_every_call(smr):
    """Route, align and both products in turn on one workspace: what one leaves
    behind means nothing to the next."""
    ws = smr.Workspace(64 << 20)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    refs = {}
    for turn in range(3):
        for T, E in ((4, 512), (16, 64), (300, 64)):
            g.manual_seed(T)
            x, gate = _normal(g, T, 256), _normal(g, E, 256, std=0.1)
            w13, w2 = _normal(g, E, 128, 256, std=0.1), _normal(g, E, 256, 64, std=0.2)
            ids, wts, *al = smr.route_align(x, gate, topk=4, block_size=64, workspace=ws)
            act = smr.expert_up(x, w13, *al, width=4, block_size=64, workspace=ws)
            out = smr.expert_down(act, w2, ids, wts, *al, block_size=64, workspace=ws)
            got = (ids, wts, act, out)
            ref = refs.setdefault(T, got)
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert smr.get_device_error(ws) == 0


@pytest.mark.parametrize("A,T", [(64, 60), (128, 60), (128, 2000)])
def test_bad_values_stay_in_their_rows(smr, A, T):
    ids, wts, _, x, w13, w2 = _case(smr, T=T)
    al = smr.align(ids, 7, A)
    good = smr.expert_up(x, w13, *al, width=3, block_size=A)
    x = x.clone()
    x[11, 5], x[12, 3] = float("nan"), float("inf")
    act = smr.expert_up(x, w13, *al, width=3, block_size=A)
    tok = torch.arange(T * 3, device="cuda") // 3
    keep = (tok != 11) & (tok != 12)
    assert torch.equal(act[keep], good[keep]) and torch.isnan(act[tok == 11]).all()
    assert not torch.isfinite(act[tok == 12]).any()
    out = smr.expert_down(act, w2, ids, wts, *al, block_size=A)
    assert torch.isfinite(out).all(1).logical_not().nonzero().flatten().tolist() == [11, 12]


def test_not_a_number_blocks(smr):
    ids, wts, al, x, w13, w2 = _case(smr, T=60)
    x = x.clone()
    x[9, 40] = float("nan")
    codes, xs = smr.quantize_mxfp4(x)
    w, ws, wv = _weights_mx(smr, w13, True)
    act = smr.expert_up(codes, w, *al, width=3, block_size=64, x_scales=xs, w_scales=ws)
    tok = torch.arange(180, device="cuda") // 3
    assert torch.isnan(act[tok == 9]).all() and torch.isfinite(act[tok != 9]).all()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [3, 500, 3000])
def test_same_bits_twice_and_tail_ignored(smr, T, mx):
    c = _case(smr, T=T)
    a = _ffn(smr, c, mx)
    n = int(c[2][2])
    c[2][0][n:] = torch.randint(0, T * 3, (c[2][0].numel() - n,), device="cuda", dtype=torch.int32)
    c[2][1][n // 64:] = 3
    b = _ffn(smr, c, mx)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_corrupted_align_outputs(smr):
    """Entries that are neither slots nor the sentinel, experts that do not
    exist and lengths past the arrays are flagged and skipped."""
    ids, wts, al, x, w13, w2 = _case(smr, T=100)
    good = smr.expert_up(x, w13, *al, width=3, block_size=64)
    srt, eids, npp = (t.clone() for t in al)
    bad_slot = int(srt[1])
    srt[1] = 1 << 29
    ws = smr.Workspace(256)
    out = torch.zeros_like(good)
    smr.expert_up(x, w13, srt, eids, npp, width=3, block_size=64, out=out, workspace=ws)
    assert smr.get_device_error(ws) == 4
    keep = torch.arange(300, device="cuda") != bad_slot
    assert torch.equal(out[keep], good[keep]) and (out[bad_slot] == 0).all()
    srt = al[0].clone()
    srt[2] = -5
    eids[0] = 7
    ws = smr.Workspace(256)
    smr.expert_up(x, w13, srt, eids, npp, width=3, block_size=64, workspace=ws)
    assert smr.get_device_error(ws) == 5
    for n in (1 << 30, -64):
        ws = smr.Workspace(256)
        npp.fill_(n)
        srt, eids = al[0].clone(), al[1].clone()
        srt[int(al[2]):] = 300
        eids[int(al[2]) // 64:] = 0
        out = torch.zeros_like(good)
        smr.expert_up(x, w13, srt, eids, npp, width=3, block_size=64, out=out, workspace=ws)
        assert smr.get_device_error(ws) == 0
        assert torch.equal(out, good if n > 0 else torch.zeros_like(good))


def test_offsets_past_32_bits(smr):
    """Outputs and rows of more than 2^31 elements (and 2^32 bytes)."""
    T, I, H = 140000, 16384, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    wts = torch.rand(T, 1, device="cuda", generator=g)
    al = smr.align(ids, 1, 128)
    x, w = _normal(g, T, H), _normal(g, 1, 2 * I, H, std=0.5)
    act = smr.expert_up(x, w, *al, width=1, block_size=128)
    rows = torch.tensor([0, 1, 65536, 131071, 131072, 131073, T - 1], device="cuda")
    one = torch.zeros(rows.numel(), 1, dtype=torch.int32, device="cuda")
    _close(act[rows], *_ref_up(x[rows].double(), w.double(), one, 1))
    w2 = _normal(g, 1, H, I, std=I ** -0.5)
    out = smr.expert_down(act, w2, ids, wts, *al, block_size=128)
    _close(out[rows], *_ref_down(act[rows].double(), w2.double(), one, wts[rows]))
    del act, out
    w2 = _normal(g, 1, I, H, std=0.25)  # the rows before the sum: T * 16384
    out = smr.expert_down(x, w2, ids, wts, *al, block_size=128)
    _close(out[rows], *_ref_down(x[rows].double(), w2.double(), one, wts[rows]))


def test_empty_batch(smr):
    al = smr.align(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 4, 64)
    w13 = torch.zeros(4, 32, 64, dtype=torch.bfloat16, device="cuda")
    act = smr.expert_up(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), w13, *al, width=2, block_size=64)
    assert act.shape == (0, 16) and smr.last_launch_count() == 0
    out = smr.expert_down(act, torch.zeros(4, 64, 16, dtype=torch.bfloat16, device="cuda"),
                          torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 2, device="cuda"),
                          *al, block_size=64)
    assert out.shape == (0, 64) and smr.last_launch_count() == 0


def test_given_outputs_and_launches(smr):
    c = _case(smr, T=9)
    ids, wts, al, x, w13, w2 = c
    ref = _ffn(smr, c)
    act, out = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    assert smr.expert_up(x, w13, *al, width=3, block_size=64, out=act) is act and smr.last_launch_count() == 1
    assert smr.expert_down(act, w2, ids, wts, *al, block_size=64, out=out) is out and smr.last_launch_count() == 2
    assert torch.equal(act, ref[0]) and torch.equal(out, ref[1])
    with pytest.raises(ValueError, match="out must be"):
        smr.expert_up(x, w13, *al, width=3, block_size=64, out=act[:-1])
    with pytest.raises(ValueError, match="one device"):
        smr.expert_up(x, w13.cpu(), *al, width=3, block_size=64)
    with pytest.raises(smr.SmrUnsupported, match="64 or 128"):
        smr.expert_up(x, w13, *al, width=3, block_size=256)
    with pytest.raises(smr.SmrError, match="16-byte aligned"):
        smr.expert_up(torch.zeros(9, 264, dtype=torch.bfloat16, device="cuda")[:, 4:260], w13, *al, width=3, block_size=64)


@pytest.mark.parametrize("K", [128, 256, 512])
@pytest.mark.parametrize("shift", [0, 4, 8])
@pytest.mark.parametrize("T", [20, 600])
def test_scale_rows_of_any_alignment(smr, K, shift, T):
    """Rows of scales that can be read 16, 8 or only 4 bytes at a time."""
    ids, _, al, x, w13, _ = _case(smr, T=T, H=K)
    w, ws = _laid_out(smr, w13, True)
    codes, xs = smr.quantize_mxfp4(x)
    ref = smr.expert_up(codes, w, *al, width=3, block_size=64, x_scales=xs, w_scales=ws)
    buf = torch.full((xs.numel() + shift,), 255, dtype=torch.uint8, device="cuda")
    moved = buf[shift:].view_as(xs)
    moved.copy_(xs)
    assert torch.equal(smr.expert_up(codes, w, *al, width=3, block_size=64, x_scales=moved, w_scales=ws), ref)
    xv, wv = smr.dequantize_mxfp4(codes, xs).double(), _mx_exact(w13)[2]
    _close(ref, *_ref_up(xv, wv, ids, 3))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,E,width,H", [
    (1, 1, 1, 16),        # one slot, one partial tile
    (2, 3, 6, 272),       # a token's slots on the same expert several times
    (16, 2, 40, 640),     # more than 32 slots a token
    (16, 300, 11, 4096),
    (7, 40, 4, 16384),    # 128 weight tiles
])
def test_down_of_few_tokens(smr, mx, T, E, width, H):
    I = 256
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)
    ids = torch.randint(0, E, (T, width), generator=g, device="cuda").int()
    if E > 2 and T > 1:
        ids[1, 0], ids[0] = -1, E  # a slot, and a whole token, that no expert has
    wts = torch.rand(T, width, generator=g, device="cuda") - 0.3
    al = smr.align(ids, E, 64, workspace=smr.Workspace(256))
    x, w = _normal(g, T * width, I), _normal(g, E, H, I, std=I ** -0.5)
    skipped = ((ids < 0) | (ids >= E)).reshape(-1)
    xa, kw, xv = _values(smr, x, mx)
    if mx:
        wa, kw["w_scales"], wv = _weights_mx(smr, w, False)
    else:
        wa, wv = w, w.double()
        xa = xa.clone()
        xa[skipped] = float("nan")  # never read
    ws = smr.Workspace(256)
    out = smr.expert_down(xa, wa, ids, wts, *al, block_size=64, workspace=ws, **kw)
    assert smr.get_device_error(ws) == 0
    _close(out, *_ref_down(torch.where(skipped[:, None], 0.0, xv), wv, ids, wts))
    assert torch.equal(out, smr.expert_down(xa, wa, ids, wts, *al, block_size=64, workspace=ws, **kw))


def test_threads_on_one_stream(smr):
    """Calls of four threads on the default stream share its workspace."""
    import threading
    cases = [_case(smr, T=T, seed=T) for T in (3, 40, 300, 600)]
    refs = [_ffn(smr, c) for c in cases]
    torch.cuda.synchronize()
    outs = [[] for _ in cases]

    def work(k):
        outs[k] += [_ffn(smr, cases[k])[1] for _ in range(25)]

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for got, ref in zip(outs, refs):
        assert len(got) == 25 and all(torch.equal(o, ref[1]) for o in got)


def test_default_stream_by_its_pointer(smr):
    c = _case(smr, T=20)
    ref = _ffn(smr, c)
    got = _ffn(smr, c, stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_workspace_on_the_host_is_refused(smr):
    ids, wts, al, x, w13, w2 = _case(smr, T=5)
    for ws in (torch.zeros(4096, dtype=torch.uint8), smr.Workspace(4096, "cpu")):
        with pytest.raises(ValueError, match="workspace must be on"):
            smr.expert_up(x, w13, *al, width=3, block_size=64, workspace=ws)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [4, 200])  # single CTAs and pairs
def test_strongly_negative_gates(smr, mx, T):
    """Gates far outside the exponential's range beside large up values, whose
    product is an ordinary number. One value of K is not zero, so the products
    are exact and only silu(g) * u is rounded: half a step of bf16, and by the
    bounds of the intrinsics 4 + 1.2 |g| + 5 units of 2^-23 (two exponentials of
    half the argument, the quotient, the sums and products)."""
    gates = torch.tensor([0.0, -0.5, 3.0, 12.0, 90.0, 200.0, -20.0, -60.0, -87.0, -87.5, -88.5, -90.0, -95.0, -100.0,
                          -120.0, -192.0] * 2, device="cuda").to(torch.bfloat16)
    ups = torch.cat([torch.full((16,), 2.0 ** 100, device="cuda"), torch.full((16,), -1.5, device="cuda")]).to(torch.bfloat16)
    I, H = 32, 128
    w = torch.zeros(1, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    w[0, :I, 0], w[0, I:, 0] = gates, ups
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    al = smr.align(ids, 1, 64)
    xa, kw, _ = _values(smr, x, mx)
    wv = w.double()
    if mx:
        w, kw["w_scales"], wv = _weights_mx(smr, w, True)
    out = smr.expert_up(xa, w, *al, width=1, block_size=64, **kw)
    g, u = wv[0, :I, 0], wv[0, I:, 0]
    ref = (g / (1 + torch.exp(-g)) * u).expand(T, I)
    _close(out, ref, (U + (9 + 1.2 * g.abs()) * 2.0 ** -23) * ref.abs() + TINY)


def test_error_bits_survive_a_growing_workspace(smr):
    """An align's flag is still there when a later call on the workspace needs more room."""
    ids, wts, _, x, w13, w2 = _case(smr, T=50)
    ids = ids.clone()
    ids[3, 1] = -1
    ws = smr.Workspace(256)
    al = smr.align(ids, 7, 64, workspace=ws)
    act = smr.expert_up(x, w13, *al, width=3, block_size=64, workspace=ws)
    out = smr.expert_down(act, w2, ids, wts, *al, block_size=64, workspace=ws)
    assert ws.nbytes > 256 and smr.get_device_error(ws) == 1
    assert torch.isfinite(out).all()
    smr.clear_device_error(ws)
    assert smr.get_device_error(ws) == 0


def test_workspace_of_a_graph(smr):
    """A caller's workspace under capture: refused where it is too small, and
    still the graph's after an eager call made it grow."""
    small, big = _case(smr, T=30, seed=4), _case(smr, T=700, seed=5)
    ref = [t.clone() for t in _ffn(smr, small)]
    ids, wts, al, x, w13, w2 = small
    ws = smr.Workspace(256)
    with pytest.raises(smr.SmrError, match="being captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            smr.expert_down(ref[0], w2, ids, wts, *al, block_size=64, workspace=ws)
    torch.cuda.synchronize()
    assert ws.nbytes == 256
    _ffn(smr, small, workspace=ws)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs = _ffn(smr, small, workspace=ws)
    before = ws.nbytes
    _ffn(smr, big, workspace=ws)
    assert ws.nbytes > before
    others = [torch.full((before,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]  # memory that was given back would be theirs
    for t in outs:
        t.zero_()
    gr.replay()
    torch.cuda.synchronize()
    assert all((o == 7).all() for o in others)
    assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1]) and smr.get_device_error(ws) == 0


def test_errors_without_a_workspace(smr):
    """The bits of calls that were given no workspace can be read: eager ones,
    replayed ones, and after the memory of a call is gone."""
    ids, wts, al, x, w13, w2 = _case(smr, T=40)
    smr.clear_device_error()
    act, out = _ffn(smr, (ids, wts, al, x, w13, w2))
    assert smr.get_device_error() == 0
    srt = al[0].clone()
    srt[1] = 1 << 29  # neither a slot nor the sentinel
    smr.expert_up(x, w13, srt, *al[1:], width=3, block_size=64, out=act)
    assert smr.get_device_error() == 4 == smr.get_device_error(None)
    smr.clear_device_error()
    assert smr.get_device_error() == 0
    eids = al[1].clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        smr.expert_down(act, w2, ids, wts, al[0], eids, al[2], block_size=64, out=out)
    gr.replay()
    assert smr.get_device_error() == 0
    eids[0] = 99  # an expert that does not exist
    gr.replay()
    assert smr.get_device_error() == 1
    eids[0] = al[1][0]
    gr.replay()
    assert smr.get_device_error() == 1  # (sticky)
    smr.clear_device_error()
    ws = smr.Workspace(256)
    smr.expert_up(x, w13, srt, *al[1:], width=3, block_size=64, out=act, workspace=ws)
    assert smr.get_device_error(ws) == 4 and smr.get_device_error() == 4
    smr.clear_device_error()
    bad = ids.clone()
    bad[0, 0] = -1
    smr.align(bad, 7, 64)  # (the workspace that these calls share)
    assert smr.get_device_error() == 1
    smr.clear_device_error()
    assert smr.get_device_error() == 0 and smr.get_device_error(ws) == 4


def test_threads_with_one_workspace(smr):
    """Four threads on the default stream with a workspace of the caller's that
    has to grow; two of them route and align on it in between."""
    import threading
    cases = [_case(smr, T=T, seed=T) for T in (40, 300, 600, 900)]
    refs = [_ffn(smr, c) for c in cases]
    als = [tuple(t.clone() for t in smr.align(c[0], 7, 64)) for c in cases]
    torch.cuda.synchronize()
    ws, outs = smr.Workspace(256), [[] for _ in cases]

    def work(k):
        for _ in range(25):
            al = smr.align(cases[k][0], 7, 64, workspace=ws) if k % 2 else cases[k][2]
            outs[k].append((_ffn(smr, cases[k], workspace=ws)[1], al))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for got, ref, al in zip(outs, refs, als):
        assert len(got) == 25
        n = int(al[2])
        for out, a in got:
            assert torch.equal(out, ref[1])
            assert int(a[2]) == n and torch.equal(a[0][:n], al[0][:n]) and torch.equal(a[1][: n // 64], al[1][: n // 64])
    assert smr.get_device_error(ws) == 0


def test_released_workspaces(smr):
    """The memory goes back, and what was queued on it still comes out right."""
    c = _case(smr, T=5000, H=1024, I=128)
    ref = _ffn(smr, c)
    smr.release_workspaces()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    for _ in range(5):
        out = _ffn(smr, c)
        smr.release_workspaces()
        torch.full((32 << 20,), 7, dtype=torch.uint8, device="cuda")  # (may take the memory over, in order)
    torch.cuda.synchronize()
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    del out
    assert torch.cuda.memory_allocated() == before
    assert smr.expert_down(ref[0], c[5], c[0], c[1], *c[2], block_size=64).shape == ref[1].shape
    assert torch.cuda.memory_allocated() - before > 5000 * 3 * 1024 * 2
    smr.release_workspaces()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,H,I,E,S,k,A,zipf", [
    (20, 272, 256, 3, 0, 2, 64, 0.0),       # fp32 rows anyway
    (700, 4096, 128, 64, 0, 4, 64, 0.0),    # single CTAs, above 2^23 values
    (700, 4096, 128, 64, 0, 4, 128, 1.1),
    (2000, 384, 384, 5, 1, 2, 64, 0.0),     # pairs
    (1500, 640, 256, 4, 0, 2, 128, 1.1),
    (3000, 400, 128, 4, 1, 1, 64, 1.1),     # pairs, partial tiles, an odd number of them
])
def test_down_with_fp32_rows(smr, mx, T, H, I, E, S, k, A, zipf):
    """Without the rounding of the rows: |do| <= sum_s |w_s| c ad_s (1 + u) +
    width 2^-24 sum_s |w_s y_s| + u |o| + 2^-134."""
    ids, wts, g = _routing(T, E, k, S, zipf, 71 + T)
    al = smr.align(ids, E + S, A)
    x, w = _normal(g, T * (k + S), I), _normal(g, E + S, H, I, std=I ** -0.5)
    xa, kw, xv = _values(smr, x, mx)
    wa, wv = w, w.double()
    if mx:
        wa, kw["w_scales"], wv = _weights_mx(smr, w, False)
    ws = smr.Workspace(256)
    out = smr.expert_down(xa, wa, ids, wts, *al, block_size=A, fp32_rows=True, workspace=ws, **kw)
    assert smr.get_device_error(ws) == 0 and smr.last_launch_count() == 2
    assert ws.nbytes >= 4 * T * (k + S) * H
    ref, _ = _ref_down(xv, wv, ids, wts)
    c = 2.0 * (I // 16 + 32) * 2.0 ** -24
    y, ad = torch.zeros(T * (k + S), H, dtype=torch.float64, device="cuda"), torch.zeros(T * (k + S), H, dtype=torch.float64, device="cuda")
    flat = ids.reshape(-1)
    for e in torch.unique(flat).tolist():
        i = torch.nonzero(flat == e).squeeze(1)
        y[i], ad[i] = xv[i] @ wv[e].T, xv[i].abs() @ wv[e].abs().T
    wt = wts.double()[:, :, None].abs()
    tol = (wt * c * ad.view(T, k + S, H)).sum(1) * (1 + U) + (k + S) * 2.0 ** -24 * (wt * y.abs().view(T, k + S, H)).sum(1)
    _close(out, ref, tol + U * ref.abs() + TINY)
    again = smr.expert_down(xa, wa, ids, wts, *al, block_size=A, fp32_rows=True, workspace=ws, **kw)
    assert torch.equal(out, again)
    if T == 20:
        assert torch.equal(out, smr.expert_down(xa, wa, ids, wts, *al, block_size=A, **kw))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    there = smr.expert_down(xa, wa, ids, wts, *al, block_size=A, fp32_rows=True, stream=s, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out, there)


def _operands(smr, x, w13, mx):
    """expert_up's operands and their 64-bit values."""
    xa, kw, xv = _values(smr, x, mx)
    if not mx:
        return xa, w13, kw, xv, w13.double()
    w, kw["w_scales"], wv = _weights_mx(smr, w13, True)
    return xa, w, kw, xv, wv


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("A", [64, 128])
def test_pairs_skipped_slots(smr, A, mx):
    """As test_skipped_slots, with enough rows an expert for CTA pairs."""
    ids, wts, _, x, w13, w2 = _case(smr, T=700)
    g = torch.Generator(device="cuda")
    g.manual_seed(A)
    ids = torch.where(torch.rand(ids.shape, device="cuda", generator=g) < 0.1, torch.full_like(ids, -1), ids)
    ids[20], ids[31, 0], ids[ids == 4] = 7, 1 << 20, -3  # a token without any, an expert without a row
    ws = smr.Workspace(256)
    al = smr.align(ids, 7, A, workspace=ws)
    assert smr.get_device_error(ws) == 1
    smr.clear_device_error(ws)
    xa, w, kw, xv, wv = _operands(smr, x, w13, mx)
    out = torch.full((2100, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    smr.expert_up(xa, w, *al, width=3, block_size=A, out=out, workspace=ws, **kw)
    gone = ((ids < 0) | (ids >= 7)).reshape(-1)
    assert (out[gone] == 5.0).all() and int((~gone).sum()) >= 48 * 7
    ref, tol = _ref_up(xv, wv, ids, 3)
    _close(out[~gone], ref[~gone], tol[~gone])
    y, kd, yv = _values(smr, torch.where(gone[:, None], torch.zeros_like(out), out), mx)
    wd, wdv = w2, w2.double()
    if mx:
        wd, kd["w_scales"], wdv = _weights_mx(smr, w2, False)
    ref, tol = _ref_down(yv, wdv, ids, wts)
    for fp32_rows in (False, True):
        z = smr.expert_down(y, wd, ids, wts, *al, block_size=A, fp32_rows=fp32_rows, workspace=ws, **kd)
        _close(z, ref, tol)
        assert (z[20] == 0).all()
    assert smr.get_device_error(ws) == 0


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("A", [64, 128])
def test_pairs_remapped_experts(smr, A, mx):
    ids, wts, _, x, w13, w2 = _case(smr, T=1200, E=6, S=0)
    phys = torch.tensor([[0, 7], [1, 1], [2, 8], [3, 3], [4, 4], [5, 6]], dtype=torch.int32, device="cuda")
    count = torch.tensor([2, 1, 2, 1, 1, 2], dtype=torch.int32, device="cuda")
    al = smr.align(ids, 6, A, eplb_map=phys, eplb_count=count, num_physical=9)
    logical = torch.tensor([0, 1, 2, 3, 4, 5, 5, 0, 2], device="cuda")
    xa, w, kw, xv, _ = _operands(smr, x, w13[logical].contiguous(), mx)
    act = smr.expert_up(xa, w, *al, width=2, block_size=A, **kw)
    _close(act, *_ref_up(xv, _mx_exact(w13)[2] if mx else w13.double(), ids, 2))
    y, kd, yv = _values(smr, act, mx)
    wd, wdv = w2[logical].contiguous(), w2.double()
    if mx:
        wd, kd["w_scales"] = _laid_out(smr, wd, False)
        wdv = _mx_exact(w2)[2]
    out = smr.expert_down(y, wd, ids, wts, *al, block_size=A, num_logical=6, **kd)
    _close(out, *_ref_down(yv, wdv, ids, wts))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("A", [64, 128])
def test_pairs_corrupted_align_outputs(smr, A, mx):
    """As test_corrupted_align_outputs, with CTA pairs: a bad entry or owner
    costs its own row or block, also in the middle of a group of blocks."""
    ids, wts, _, x, w13, w2 = _case(smr, T=900)
    al = smr.align(ids, 7, A)
    n = int(al[2])
    xa, w, kw, xv, wv = _operands(smr, x, w13, mx)
    good = smr.expert_up(xa, w, *al, width=3, block_size=A, **kw)
    _close(good, *_ref_up(xv, wv, ids, 3))
    srt, eids, npp = (t.clone() for t in al)
    real = torch.nonzero(al[0][:n] < 2700).flatten()
    hit = real[torch.tensor([1, 700, 1300, 2699], device="cuda")]
    lost = al[0][hit].long()
    srt[hit] = torch.tensor([1 << 29, -5, 2701, -(1 << 31)], dtype=torch.int32, device="cuda")
    ws = smr.Workspace(256)
    out = torch.zeros_like(good)
    smr.expert_up(xa, w, srt, eids, npp, width=3, block_size=A, out=out, workspace=ws, **kw)
    assert smr.get_device_error(ws) == 4
    keep = torch.ones(2700, dtype=torch.bool, device="cuda")
    keep[lost] = False
    assert torch.equal(out[keep], good[keep]) and (out[lost] == 0).all()
    for block, owner in ((0, 7), (1, -1), (n // A - 1, 1 << 30)):
        bad = eids.clone()
        bad[block] = owner
        ws = smr.Workspace(256)
        out = torch.zeros_like(good)
        smr.expert_up(xa, w, al[0], bad, npp, width=3, block_size=A, out=out, workspace=ws, **kw)
        assert smr.get_device_error(ws) == 1
        rows = al[0][block * A:(block + 1) * A].long()
        keep = torch.ones(2701, dtype=torch.bool, device="cuda")
        keep[rows] = False
        keep = keep[:2700]
        assert torch.equal(out[keep], good[keep]) and (out[~keep] == 0).all() and (~keep).any()
    for length in (1 << 30, -64, 0):
        ws = smr.Workspace(256)
        npp.fill_(length)
        srt, eids = al[0].clone(), al[1].clone()
        srt[n:], eids[n // A:] = 2700, 0
        out = torch.zeros_like(good)
        smr.expert_up(xa, w, srt, eids, npp, width=3, block_size=A, out=out, workspace=ws, **kw)
        assert smr.get_device_error(ws) == 0
        assert torch.equal(out, good if length > 0 else torch.zeros_like(good))


@pytest.mark.parametrize("A", [64, 128])
def test_pairs_not_a_number_blocks(smr, A):
    ids, wts, _, x, w13, w2 = _case(smr, T=800)
    al = smr.align(ids, 7, A)
    x = x.clone()
    x[9, 40], x[700, 255] = float("nan"), float("inf")
    codes, xs = smr.quantize_mxfp4(x)
    w, ws, wv = _weights_mx(smr, w13, True)
    act = smr.expert_up(codes, w, *al, width=3, block_size=A, x_scales=xs, w_scales=ws)
    tok = torch.arange(2400, device="cuda") // 3
    bad = (tok == 9) | (tok == 700)
    assert torch.isnan(act[bad]).all()
    ref, tol = _ref_up(_mx_exact(torch.where(torch.isfinite(x), x, torch.zeros_like(x)))[2], wv, ids, 3)
    _close(act[~bad], ref[~bad], tol[~bad])
    # a weight whose block is not a number: its expert's rows at its feature only
    w13 = w13.clone()
    w13[2, 128 + 17, 3] = float("nan")  # an up row
    w, ws = _laid_out(smr, w13, True)
    good = act
    act = smr.expert_up(codes, w, *al, width=3, block_size=A, x_scales=xs, w_scales=ws)
    of2 = (ids == 2).reshape(-1) & ~bad
    assert torch.isnan(act[of2, 17]).all() and of2.any()
    act[of2, 17] = good[of2, 17]
    assert torch.equal(act[~bad], good[~bad])
    y, yx = smr.quantize_mxfp4(good)
    w, ws = _laid_out(smr, w2, False)
    out = smr.expert_down(y, w, ids, wts, *al, block_size=A, x_scales=yx, w_scales=ws)
    assert torch.isnan(out).all(1).nonzero().flatten().tolist() == [9, 700]
    assert torch.isfinite(out).all(1).logical_not().nonzero().flatten().tolist() == [9, 700]


@pytest.mark.parametrize("mx", [False, True])
def test_streams_with_their_own_inputs(smr, mx):
    """Calls without a workspace on several streams at once, each stream with
    other inputs and sizes: none reads another's rows."""
    cases = [_case(smr, T=T, H=1024, seed=T) for T in (900, 1100, 1500, 2000)]
    refs = [_ffn(smr, c, mx) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[] for _ in cases]
    for _ in range(12):
        for c, s, o in zip(cases, streams, outs):
            o.append(_ffn(smr, c, mx, stream=s))
    torch.cuda.synchronize()
    for ref, o in zip(refs, outs):
        assert all(torch.equal(a, ref[0]) and torch.equal(b, ref[1]) for a, b in o)


@pytest.mark.parametrize("A,T", [(64, 40), (128, 40), (64, 1000), (128, 1000)])
def test_align_outputs_of_any_alignment(smr, A, T):
    """sorted_token_ids and expert_ids are asked to be 4-byte aligned only, and
    may end with the last block's entries."""
    ids, wts, _, x, w13, w2 = _case(smr, T=T)
    al = smr.align(ids, 7, A)
    ref = smr.expert_up(x, w13, *al, width=3, block_size=A)
    n = int(al[2])
    last = int((al[0][:n] < 3 * T).nonzero()[-1]) + 1  # (the sentinels behind the last slot may be missing)
    for shift in (0, 1, 2, 3):
        srt = torch.full((shift + last,), -1, dtype=torch.int32, device="cuda")[shift:]
        eids = torch.full((shift + n // A,), -1, dtype=torch.int32, device="cuda")[shift:]
        srt.copy_(al[0][:last])
        eids.copy_(al[1][: n // A])
        ws = smr.Workspace(256)
        out = torch.full_like(ref, float("nan"))
        smr.expert_up(x, w13, srt, eids, al[2], width=3, block_size=A, out=out, workspace=ws)
        assert smr.get_device_error(ws) == 0 and torch.equal(out, ref)
    _close(ref, *_ref_up(x.double(), w13.double(), ids, 3))
