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


def _weights_mx(smr, w, gated):
    codes, scales = smr.quantize_mxfp4(w)
    return codes, smr.tile_mxfp4_scales(scales, gated=gated), _mx_exact(w)[2]


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
]
SHAPES_MX = [
    (1, 128, 128, 1, 0, 1, 64, 0.0),
    (1, 2048, 768, 128, 0, 8, 64, 0.0),
    (5, 384, 384, 6, 1, 2, 64, 0.0),      # K % 256 = 128: half a k-block
    (40, 256, 128, 3, 0, 2, 128, 0.0),
    (300, 512, 256, 64, 1, 8, 64, 1.1),
    (1000, 256, 640, 16, 0, 4, 128, 2.0),
]


@pytest.mark.parametrize("mx,shape", [(False, s) for s in SHAPES] + [(True, s) for s in SHAPES_MX])
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


@pytest.mark.parametrize("mx,shape", [(False, s) for s in SHAPES] + [(True, s) for s in SHAPES_MX])
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
