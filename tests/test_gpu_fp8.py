"""The experts' products on E4M3 operands with one fp32 scale per 128 values
(weights: per 128 x 128 block), and the format's quantisation, against plain
64-bit forms. Needs a GB300.

The products' bounds are those of test_gpu_ffn with c = 2 (K/16 + 32) 2^-24: a
block of 128 takes four updates of the accumulator, then one rounding of the
scales' product, one of their product with the row's, and one of the sum, fewer
than one rounding per 16 values and 32 more.
"""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_ffn import _close, _normal, _ref_down, _ref_up, _routing, smr  # noqa: E402, F401

BLOCK = 128


def _e4m3(v):
    """v (64 bits) to the nearest E4M3 value, ties to the even code, saturated."""
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / unit) * unit).clamp(-448, 448)


def _quant_ref(b, dims):
    """(values of the codes, scales) of blocks: the definition, each 32-bit operation rounded once from 64 bits."""
    b = b.double()
    amax = b.abs().amax(dims, keepdim=True)
    some, bad = amax > 0, ~torch.isfinite(amax)
    top = torch.where(some & ~bad, amax.clamp(min=2.0 ** -110), torch.ones_like(amax))
    scale = torch.where(some, (top / 448).float().double(), torch.zeros_like(top))
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    v = (b * (448 / top).float().double()).float().double()
    return torch.where(some & ~bad, _e4m3(torch.where(bad, torch.zeros_like(v), v)), torch.zeros_like(v)), scale


def _rows_ref(x):
    """Codes' values [..., K] and scales [..., ceil(K / 128)] of rows."""
    K = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    q, s = _quant_ref(b, -1)
    return q.flatten(-2)[..., :K], s.squeeze(-1)


def _weight_ref(w, gated):
    """The same of a weight's 128 x 128 blocks; a gated one's halves apart."""
    E, N, K = w.shape
    if gated:
        q, s = _weight_ref(w.view(2 * E, N // 2, K), False)
        return q.reshape(E, N, K), s.reshape(E, -1, s.shape[-1])
    b = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK)).unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))
    q, s = _quant_ref(b, (-1, -3))
    return q.flatten(-2).flatten(-3, -2)[:, :N, :K], s.squeeze(-1).squeeze(-2)


def _row_values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double()
    return v * scales.double().repeat_interleave(BLOCK, -1)[..., : v.shape[-1]]


def _weight_values(codes, scales, gated):
    E, N, K = codes.shape
    if gated:
        return _weight_values(codes.view(2 * E, N // 2, K), scales.view(2 * E, -1, scales.shape[-1]), False).view(E, N, K)
    return _row_values(codes, scales.repeat_interleave(BLOCK, -2)[:, :N])


def _same(got, ref):
    assert torch.equal(torch.nan_to_num(got.double(), nan=7e30), torch.nan_to_num(ref.double(), nan=7e30))


# ------------------------------------------------------------- the format --

@pytest.mark.parametrize("rows,K", [(1, 32), (1, 128), (3, 160), (17, 2048), (70, 96), (1000, 4096), (4099, 352)])
def test_quantize_is_the_definition(smr, rows, K):
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    x = _normal(g, rows, K) * torch.exp2(torch.randint(-20, 20, (rows, 1), device="cuda", generator=g)).to(torch.bfloat16)
    codes, scales = smr.quantize_fp8(x)
    q, s = _rows_ref(x)
    _same(codes.view(torch.float8_e4m3fn), q)
    _same(scales, s)
    _same(smr.dequantize_fp8(codes, scales), (q * s.repeat_interleave(BLOCK, -1)[:, :K]).float().to(torch.bfloat16))


def test_quantize_special_blocks_and_strides(smr):
    x = torch.zeros(9, 256, dtype=torch.bfloat16, device="cuda")
    x[1] = -0.0
    x[2, 5], x[2, 200] = float("nan"), 3.0
    x[3, 0] = float("inf")
    x[4, 127] = -float("inf")
    x[5, 3], x[5, 4] = 2.0 ** -133, -(2.0 ** -130)   # subnormal: far below the least scale's codes
    x[6, 3], x[6, 4] = 2.0 ** -111, 2.0 ** -119      # the least scale
    x[7] = torch.finfo(torch.bfloat16).max
    x[8, :128] = torch.arange(128, device="cuda") * 3.5  # every code, ties among them
    codes, scales = smr.quantize_fp8(x)
    q, s = _rows_ref(x)
    _same(codes.view(torch.float8_e4m3fn), q)
    _same(scales, s)
    assert not codes[:5, :128].any() and scales[2, 0].isnan() and scales[2, 1] > 0 and not scales[0].any()
    wide = torch.full((9, 320), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:] = x
    for view in (wide[:, 64:], x.view(3, 3, 256)):
        c2, s2 = smr.quantize_fp8(view)
        _same(c2.view(torch.uint8).view(9, 256), codes)
        _same(s2.view(9, 2), scales)


def test_route_writes_the_same_codes(smr):
    g = torch.Generator(device="cuda").manual_seed(4)
    for M in (5, 200):
        x, w = _normal(g, M, 256), _normal(g, 32, 256)
        codes = torch.empty(M, 256, dtype=torch.uint8, device="cuda")
        scales = torch.empty(M, 2, device="cuda")
        smr.route(x, w, topk=4, hidden_fp8=codes, hidden_scales=scales)
        c, s = smr.quantize_fp8(x)
        assert torch.equal(c, codes) and torch.equal(s, scales)


@pytest.mark.parametrize("E,N,K,gated", [(1, 16, 32, False), (3, 256, 128, False), (2, 144, 352, False), (2, 96, 160, True), (5, 512, 256, True)])
def test_quantize_weight_is_the_definition(smr, E, N, K, gated):
    g = torch.Generator(device="cuda").manual_seed(E + N)
    w = _normal(g, E, N, K)
    w[0, :5, :7] = 0
    codes, scales = smr.quantize_fp8_weight(w, gated=gated)
    q, s = _weight_ref(w, gated)
    _same(codes.view(torch.float8_e4m3fn), q)
    _same(scales, s)


def test_dequantize_every_code(smr):
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(5, 1)
    scales = torch.tensor([0.0, 1.0, 0.3, 3e-39, 1e38], device="cuda")[:, None].repeat(1, 2)
    ref = codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(BLOCK, -1)
    _same(smr.dequantize_fp8(codes, scales), ref.to(torch.bfloat16))
    _same(smr.dequantize_fp8(codes.view(torch.float8_e4m3fn), scales), ref.to(torch.bfloat16))


# ---------------------------------------------------------------- products --

# T, H, I, E, S, k, A, zipf
SHAPES = [
    (1, 32, 32, 1, 0, 1, 64, 0.0),        # one of everything
    (1, 2048, 768, 128, 0, 8, 64, 0.0),   # a single token
    (3, 96, 64, 5, 1, 2, 64, 0.0),        # partial tiles and blocks
    (16, 256, 64, 4, 0, 4, 128, 0.0),     # 16 rows: whole columns
    (17, 288, 160, 7, 0, 3, 128, 0.0),    # one row more than 16
    (65, 160, 192, 3, 1, 2, 64, 0.0),     # a second block of one row
    (130, 640, 384, 3, 0, 2, 128, 0.0),   # five and three k-blocks
    (300, 512, 192, 64, 1, 8, 64, 1.1),
    (1000, 256, 128, 16, 0, 4, 128, 2.0),  # hot experts over many blocks
    (2500, 128, 96, 6, 1, 3, 64, 0.0),
    (4000, 416, 224, 5, 0, 2, 128, 0.0),  # pairs of CTAs: whole and partial tiles and k-blocks
    (3000, 288, 352, 4, 1, 1, 64, 1.1),   # pairs, an odd number of weight tiles, groups of blocks
    (2000, 1152, 768, 4, 0, 2, 128, 0.0),
]


def _uneven(g, x, dim):
    """Blocks of very different size: every scale counts."""
    n = -(-x.shape[dim] // BLOCK)
    f = torch.exp2(torch.randint(-4, 5, (n,), device="cuda", generator=g).float()).repeat_interleave(BLOCK)[: x.shape[dim]]
    shape = [1] * x.dim()
    shape[dim] = -1
    return (x.float() * f.view(shape)).to(torch.bfloat16)


def _up_case(smr, shape, seed=11):
    T, H, I, E, S, k, A, zipf = shape
    ids, wts, g = _routing(T, E, k, S, zipf, seed + T)
    al = smr.align(ids, E + S, A)
    x = _uneven(g, _normal(g, T, H), 1)
    w = _uneven(g, _normal(g, E + S, 2 * I, H, std=0.3 * H ** -0.5), 1)
    xc, xs = smr.quantize_fp8(x)
    wc, ws = smr.quantize_fp8_weight(w, gated=True)
    return ids, wts, g, al, (xc, xs), (wc, ws)


@pytest.mark.parametrize("shape", SHAPES + [(40, 256, 80, 3, 0, 2, 64, 0.0), (900, 288, 176, 4, 1, 1, 128, 0.0)])
def test_up_matches_64_bits(smr, shape):
    T, H, I, E, S, k, A, zipf = shape
    ids, _, _, al, (xc, xs), (wc, wsc) = _up_case(smr, shape)
    out = torch.full((T * (k + S), I), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = smr.Workspace()
    smr.expert_up(xc, wc, *al, width=k + S, block_size=A, out=out, workspace=ws, x_scales=xs, w_scales=wsc)
    assert smr.get_device_error(ws) == 0 and smr.last_launch_count() == 1
    _close(out, *_ref_up(_row_values(xc, xs), _weight_values(wc, wsc, True), ids, k + S))


@pytest.mark.parametrize("fp32_rows", [False, True])
@pytest.mark.parametrize("shape", SHAPES + [(40, 80, 256, 3, 0, 2, 64, 0.0), (900, 176, 288, 4, 1, 1, 128, 0.0)])
def test_down_matches_64_bits(smr, shape, fp32_rows):
    T, H, I, E, S, k, A, zipf = shape
    ids, wts, g = _routing(T, E, k, S, zipf, 31 + T)
    al = smr.align(ids, E + S, A)
    xc, xs = smr.quantize_fp8(_uneven(g, _normal(g, T * (k + S), I), 1))
    wc, wsc = smr.quantize_fp8_weight(_uneven(g, _normal(g, E + S, H, I, std=I ** -0.5), 1))
    ws = smr.Workspace()
    out = smr.expert_down(xc, wc, ids, wts, *al, block_size=A, workspace=ws, x_scales=xs, w_scales=wsc, fp32_rows=fp32_rows)
    assert smr.get_device_error(ws) == 0 and smr.last_launch_count() == 2
    _close(out, *_ref_down(_row_values(xc, xs), _weight_values(wc, wsc, False), ids, wts))


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[2] % 32 == 0])
def test_quantized_act_is_that_of_two_calls(smr, shape):
    T, H, I, E, S, k, A, zipf = shape
    ids, _, _, al, (xc, xs), (wc, wsc) = _up_case(smr, shape)
    kw = dict(width=k + S, block_size=A, x_scales=xs, w_scales=wsc)
    act = smr.expert_up(xc, wc, *al, **kw)
    ws = smr.Workspace()
    codes, scales = smr.expert_up(xc, wc, *al, quantize_act=True, workspace=ws, **kw)
    assert smr.get_device_error(ws) == 0
    c, s = smr.quantize_fp8(act)
    assert torch.equal(codes, c) and torch.equal(scales, s)
