"""GPU parity of the RMS norm with the residual's addition and of its
gradients against float64.

Tolerances, u = 2^-24. A row sum of d values is formed in fp32 by at most
max(32, d/128) sequential additions a thread and 10 more in the two shuffle
trees: relative error E = (max(32, d/128) + 12) u of a sum of squares, half of
it in rstd, plus four roundings. y adds two products and the bf16 half step
2^-8. Codes are off by half a step of theirs (2^-4 of the value, 2^-10 below
the normal range) plus what y and the scale are off.
"""

import numpy as np
import pytest
import torch

from oracle import fp8, norm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
WIDTHS = [(1, 1), (3, 7), (70, 8), (2, 64), (1300, 4104), (1300, 2501), (5, 128), (9, 129), (700, 256), (33, 264), (4, 1000), (257, 1024), (3, 4096), (150, 4099),
          (2, 8192), (2, 12344), (3, 16385), (2, 20000), (2, 33000), (3, 40001)]


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


def _inputs(rows, d, seed):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    x, res = t(rows, d), t(rows, d)
    x[:, ::37] *= 30
    return x.bfloat16().cuda(), res.bfloat16().cuda(), (1 + 0.3 * t(d)).bfloat16().cuda(), rng


def _np(t):
    return t.double().cpu().numpy()


def _rel(d):
    return (max(32, d / 128) + 12) * U / 2 + 4 * U


@pytest.mark.parametrize("rows,d", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(q, rows, d, residual):
    x, res, gamma, _ = _inputs(rows, d, rows + d)
    x0, eps = x.clone(), 1e-5
    y, h, rstd = q.qlora_rmsnorm_fwd(x, gamma, eps, residual=res if residual else None)
    want_h = (x.float() + res.float()).bfloat16() if residual else x0
    assert torch.equal(h, want_h) and torch.equal(x, x0)
    ry, rr = norm.forward(_np(want_h), _np(gamma), float(np.float32(eps)))
    assert np.all(np.abs(_np(rstd) - rr) <= _rel(d) * rr)
    assert np.all(np.abs(_np(y) - ry) <= (2.0 ** -8 * (1 + 2.0 ** -8) + _rel(d) + 3 * U) * np.abs(ry) + 2.0 ** -134)
    for fmt in (q.FP8_E4M3, q.FP8_E5M2):
        f = fp8.FORMATS[fmt]
        y8, h8, rstd8 = q.qlora_rmsnorm_fwd(x, gamma, eps, residual=res if residual else None, fp8=True, fmt=fmt)
        assert torch.equal(h8, h) and torch.equal(rstd8, rstd)
        nb = -(-d // 128)
        wide = np.zeros((rows, nb * 128))
        wide[:, :d] = ry
        scale = np.maximum(np.abs(wide.reshape(rows, nb, 128)).max(2), 2.0 ** -100) / f["top"]
        rel = _rel(d) + 6 * U
        assert np.all(np.abs(_np(y8.scales) - scale) <= rel * scale)
        c = ry / np.repeat(scale, 128, 1)[:, :d]
        codes = fp8.decode(y8.codes.contiguous().view(torch.uint8).cpu().numpy(), f)
        half = np.maximum(2.0 ** -(f["mant"] + 1) * np.abs(c), 2.0 ** (f["emin"] - f["mant"] - 1))
        assert np.all(np.abs(codes - c) <= half * (1 + 2.0 ** -f["mant"]) + 2 * rel * np.abs(c) + 1e-30)


def test_forward_in_place_and_out_buffers(q):
    x, res, gamma, _ = _inputs(37, 520, 1)
    y, h, rstd = q.qlora_rmsnorm_fwd(x, gamma, residual=res)
    for which in (0, 1):                      # h into x's or the residual's own buffer
        a, b = x.clone(), res.clone()
        y2, h2, _ = q.qlora_rmsnorm_fwd(a, gamma, residual=b, h=(a, b)[which])
        assert torch.equal(y2, y) and torch.equal(h2, h) and h2 is (a, b)[which]
    wide = [_inputs(2, 40000, 2)[i] for i in range(3)]
    y, h, _ = q.qlora_rmsnorm_fwd(wide[0], wide[2], residual=wide[1])
    a = wide[0].clone()
    y2, h2, _ = q.qlora_rmsnorm_fwd(a, wide[2], residual=wide[1], h=a)
    assert torch.equal(y2, y) and torch.equal(a, h)
    big = torch.full((40, 520), 5.0, dtype=torch.bfloat16, device="cuda")
    out, _, _ = q.qlora_rmsnorm_fwd(x, gamma, y=big[:37])
    assert torch.equal(out, q.qlora_rmsnorm_fwd(x, gamma)[0]) and torch.all(big[37:] == 5.0)
    with pytest.raises(ValueError):
        q.qlora_rmsnorm_fwd(x[:, 1:], gamma[1:])          # not contiguous
    with pytest.raises(ValueError):
        q.qlora_rmsnorm_fwd(x, gamma, h=res)              # h without a residual
    with pytest.raises(ValueError):
        q.qlora_rmsnorm_fwd(x, gamma.float())
    with pytest.raises(q.QloraError):
        q.qlora_rmsnorm_fwd(x.view(-1)[1:521].view(1, 520), gamma)   # not 16-byte aligned
    empty = torch.empty(0, 520, dtype=torch.bfloat16, device="cuda")
    assert q.qlora_rmsnorm_fwd(empty, gamma)[0].shape == (0, 520)


def test_rows_of_zeros_and_values_that_are_not_finite(q):
    x, _, gamma, _ = _inputs(6, 264, 3)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 6] = float("inf")
    x[4] *= 1e-30
    y, _, rstd = q.qlora_rmsnorm_fwd(x, gamma, 1e-6)
    assert torch.all(y[1] == 0) and torch.all(torch.isfinite(y[[0, 1, 4, 5]]))
    assert torch.all(torch.isnan(y[2])) and rstd[3] == 0 and torch.isnan(y[3, 6])
    y8, _, _ = q.qlora_rmsnorm_fwd(x, gamma, 1e-6, fp8=True)
    v = y8.dequantize()
    assert torch.all(v[1] == 0) and torch.all(torch.isfinite(v[[0, 1, 4, 5]])) and torch.all(torch.isfinite(y8.scales))
    assert torch.all(torch.isnan(v[2])) and torch.isnan(v[3, 6])


@pytest.mark.parametrize("rows,d", WIDTHS + [(1100, 136), (900, 1000)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward(q, rows, d, residual):
    h, dres, gamma, rng = _inputs(rows, d, rows * 3 + d)
    dy = torch.from_numpy(rng.standard_normal((rows, d)).astype(np.float32) * 0.1).bfloat16().cuda()
    rstd = q.qlora_rmsnorm_fwd(h, gamma, 1e-5)[2]
    dx, dgamma = q.qlora_rmsnorm_bwd(dy, h, gamma, rstd, dres=dres if residual else None)
    hn, dyn, gn, rn = _np(h), _np(dy), _np(gamma), _np(rstd)
    rdx, rdg = norm.backward(dyn, hn, gn, rn, _np(dres) if residual else None)
    # terms of dx: dy g rstd (three roundings), h c rstd (c off by the row sum's error against the
    # sum of magnitudes, and six roundings), dres; each sum rounds once more
    up = np.abs(dyn * gn)
    c_abs = np.mean(up * np.abs(hn), axis=1) * rn ** 2
    terms = (up + np.abs(hn) * c_abs[:, None]) * rn[:, None]
    e = (max(32, d / 64) + 20) * U
    extra = np.abs(_np(dres)) if residual else 0
    assert np.all(np.abs(_np(dx) - rdx) <= 2.0 ** -8 * np.abs(rdx) + e * (terms + extra) * (1 + 2.0 ** -8) + 2.0 ** -134)
    s = np.sum(np.abs(dyn * hn * rn[:, None]), axis=0)
    assert np.all(np.abs(_np(dgamma) - rdg) <= (rows + 8) * U * s)
    again = q.qlora_rmsnorm_bwd(dy, h, gamma, rstd, dres=dres if residual else None)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dgamma)      # bit for bit
    only, none = q.qlora_rmsnorm_bwd(dy, h, gamma, rstd, dres=dres if residual else None, want_dgamma=False)
    assert none is None and torch.equal(only, dx)


def test_backward_in_place_no_rows_and_workspace(q):
    h, dres, gamma, _ = _inputs(50, 1000, 9)
    dy = dres.clone() * 0.5
    rstd = q.qlora_rmsnorm_fwd(h, gamma)[2]
    dx, dg = q.qlora_rmsnorm_bwd(dy, h, gamma, rstd, dres=dres)
    a = dres.clone()
    assert q.qlora_rmsnorm_bwd(dy, h, gamma, rstd, dres=a, dx=a)[0] is a and torch.equal(a, dx)
    b = dy.clone()
    assert torch.equal(q.qlora_rmsnorm_bwd(b, h, gamma, rstd, dres=dres, dx=b)[0], dx)
    ws = torch.empty(q.qlora_rmsnorm_workspace_bytes(50, 1000), dtype=torch.uint8, device="cuda")
    assert torch.equal(q.qlora_rmsnorm_bwd(dy, h, gamma, rstd, dres=dres, ws=ws)[1], dg)
    with pytest.raises(q.QloraError):
        q.qlora_rmsnorm_bwd(dy, h, gamma, rstd, ws=ws[:-16])
    empty = torch.empty(0, 1000, dtype=torch.bfloat16, device="cuda")
    out = torch.full((1000,), 3.0, device="cuda")
    dx, dg = q.qlora_rmsnorm_bwd(empty, empty, gamma, torch.empty(0, device="cuda"), dgamma=out)
    assert dx.shape == (0, 1000) and torch.all(out == 0)


def test_gradient_against_differences(q):
    # differences of the kernel's own forward along one direction, in the values
    # that bf16 holds: x + t, x - t with t a power of two, exact for these x
    g = torch.Generator().manual_seed(4)
    rows, d, t = 4, 96, 2.0 ** -3
    x = (torch.randint(4, 8, (rows, d), generator=g) * torch.where(torch.rand(rows, d, generator=g) < 0.5, -1, 1)).bfloat16().cuda()
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    dy = torch.randn(rows, d, generator=g).bfloat16().cuda()
    v = torch.where(torch.rand(rows, d, generator=g) < 0.5, -1.0, 1.0).cuda()
    y, h, rstd = q.qlora_rmsnorm_fwd(x, gamma, 0.0)
    dx, _ = q.qlora_rmsnorm_bwd(dy, h, gamma, rstd)
    up, down = (q.qlora_rmsnorm_fwd((x.float() + s * t * v).bfloat16(), gamma, 0.0)[0].double() for s in (1, -1))
    diff = ((up - down) * dy.double()).sum() / (2 * t)
    slope = (dx.double() * v.double()).sum()
    # y off by half a bf16 step at either end, dx by half a step; third order of the difference below 4 t^2 of it
    scale = (y.double().abs() * dy.double().abs()).sum()
    assert abs(diff - slope) <= 2.0 ** -8 * scale / t + 2.0 ** -8 * dx.double().abs().sum() + 4 * (t / 5.5) ** 2 * scale


def test_captured_and_on_another_stream(q):
    x, res, gamma, _ = _inputs(20, 512, 6)
    want = q.qlora_rmsnorm_fwd(x, gamma, residual=res, fp8=True)
    bwant = q.qlora_rmsnorm_bwd(res, want[1], gamma, want[2], dres=x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, h, r = q.qlora_rmsnorm_fwd(x, gamma, residual=res, fp8=True)
        b = q.qlora_rmsnorm_bwd(res, h, gamma, r, dres=x)
    for _ in range(2):
        h.zero_()
        g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, h2, r2 = q.qlora_rmsnorm_fwd(x, gamma, residual=res, fp8=True, stream=side)
    b2 = q.qlora_rmsnorm_bwd(res, h2, gamma, r2, dres=x, stream=side)
    torch.cuda.synchronize()
    for yy, hh, rr, bb in ((y, h, r, b), (y2, h2, r2, b2)):
        assert torch.equal(yy.codes.view(torch.uint8), want[0].codes.view(torch.uint8)) and torch.equal(yy.scales, want[0].scales)
        assert torch.equal(hh, want[1]) and torch.equal(rr, want[2])
        assert torch.equal(bb[0], bwant[0]) and torch.equal(bb[1], bwant[1])


def test_offsets_past_31_bits(q):
    d = 8192
    rows = 2 ** 31 // d + 1300
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda").normal_()
    gamma = torch.rand(d, device="cuda").bfloat16()
    tail = x[-1300:].clone()
    y, _, rstd = q.qlora_rmsnorm_fwd(x, gamma)
    y8, _, _ = q.qlora_rmsnorm_fwd(x, gamma, fp8=True)
    dx, _ = q.qlora_rmsnorm_bwd(y, x, gamma, rstd, want_dgamma=False)
    # rows do not depend on one another (as many as take the same sum's order)
    ty, _, trstd = q.qlora_rmsnorm_fwd(tail, gamma)
    ty8, _, _ = q.qlora_rmsnorm_fwd(tail, gamma, fp8=True)
    tdx, _ = q.qlora_rmsnorm_bwd(ty, tail, gamma, trstd, want_dgamma=False)
    assert torch.equal(y[-1300:], ty) and torch.equal(rstd[-1300:], trstd) and torch.equal(dx[-1300:], tdx)
    assert torch.equal(y8.codes[-1300:].view(torch.uint8), ty8.codes.view(torch.uint8))
    assert torch.equal(y8.scales[-1300:], ty8.scales)
