"""GPU parity of the 8-bit linear: quantizers bit-exact with the oracle,
products within the rounding that their arithmetic allows.

Tolerance of a product element with reduction length R and S = sum |x| |w|
(values with their scales): at most 128 fp32 additions within a block, each
off by at most 2^-23 of the running magnitude (additions of a tensor core may
truncate), two roundings for the scales, one addition per block, then one
rounding to bf16 (half a step: 2^-8):
    |y - ref| <= 2^-8 |ref| + (128 + ceil(R/128) + 4) 2^-23 S, and a bf16 subnormal's half step
"""

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu

TDTYPE = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


def _u8(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _same_codes(got, want):
    # zero has two codes; everything else has to be equal
    got, want = (np.where((c & 0x7F) == 0, 0, c) for c in (got, want))
    return np.array_equal(got, want)


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * scale).bfloat16()


def _check_product(got, x, w):
    """x [m, R], w [c, R] fp64 values."""
    ref, s = x @ w.T, np.abs(x) @ np.abs(w).T
    r = x.shape[1]
    tol = 2.0 ** -8 * np.abs(ref) + (128 + -(-r // 128) + 4) * 2.0 ** -23 * s + 2.0 ** -134
    off = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(off <= tol), (np.max(off / tol), np.unravel_index(np.argmax(off / tol), off.shape))


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 127), (5, 128), (4, 129), (33, 1000), (2, 4099), (7, 8192), (2, 40000)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_rows_bit_exact(q, rows, cols, fmt):
    rng = np.random.default_rng(rows * cols)
    x = _bf16(rng, rows, cols) * torch.exp2(torch.from_numpy(rng.integers(-12, 12, (rows, cols)))).bfloat16()
    if rows > 2:
        x[0] = 0                                     # a block of zeros
        x[1, :min(cols, 200)] = float("nan")         # blocks with nothing finite
        x[2, -1] = float("-inf")
    out = q.qlora_quantize_fp8_rows(x.cuda(), fmt=fmt)
    codes, scales = fp8.quantize_rows(x.float().numpy(), fp8.FORMATS[fmt])
    assert np.array_equal(out.scales.cpu().numpy(), scales)
    assert _same_codes(_u8(out.codes), codes)


def test_quantize_rows_extremes_and_padding(q):
    # largest and smallest values of bf16; bytes past a row's end stay as they were
    x = torch.tensor([[3.38e38, 1e-38, -3.38e38, 1.0] * 5, [1e-38, -9e-41, 0.0, 2e-39] * 5]).bfloat16()
    raw = torch.full((2, 32), 0x55, dtype=torch.uint8, device="cuda")
    rows = q.FP8Rows(raw.view(torch.float8_e4m3fn)[:, :20], torch.zeros(2, 1, device="cuda"))
    q.qlora_quantize_fp8_rows(x.cuda(), out=rows)
    codes, scales = fp8.quantize_rows(x.float().numpy(), fp8.E4M3)
    assert np.array_equal(rows.scales.cpu().numpy(), scales)
    assert _same_codes(_u8(rows.codes), codes)
    assert torch.all(raw[:, 20:] == 0x55)


@pytest.mark.parametrize("n,k", [(1, 16), (128, 128), (130, 272), (257, 1040), (1000, 512)])
def test_quantize_weight_bit_exact(q, n, k):
    rng = np.random.default_rng(n + k)
    w = _bf16(rng, n, k, scale=0.02)
    if n > 129:
        w[:128, :128] = 0
        w[129, 3] = float("nan")
    qw = q.qlora_quantize_fp8(w.cuda())
    codes, scales = fp8.quantize_weight(w.float().numpy())
    assert np.array_equal(qw.scales.cpu().numpy(), scales)
    assert _same_codes(_u8(qw.codes), codes)
    back = q.qlora_dequantize_fp8(qw).float().cpu()
    want = torch.from_numpy((fp8.decode(codes, fp8.E4M3).astype(np.float32) *
                             np.repeat(np.repeat(scales, 128, 0), 128, 1)[:n, :k])).bfloat16().float()
    assert torch.equal(torch.nan_to_num(back, 7.0), torch.nan_to_num(want, 7.0))


SHAPES = [(1, 64, 64), (3, 1003, 1040), (4, 520, 4112), (4, 1000, 272), (5, 264, 1040), (1, 1, 16), (2, 4096, 4096), (8, 1003, 1040), (9, 257, 272), (16, 384, 4096), (17, 130, 4112),
          (33, 1000, 512), (64, 11008, 1024), (127, 129, 144), (128, 256, 128), (129, 512, 640), (200, 4096, 1024),
          (256, 256, 256), (257, 1003, 1040), (300, 264, 2064), (513, 777, 1296), (1000, 2048, 512), (1300, 2307, 272), (1300, 2306, 272), (2100, 1500, 1296), (600, 5000, 1040)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forward(q, m, n, k):
    rng = np.random.default_rng(m * 31 + n + k)
    codes, scales = fp8.quantize_weight(rng.standard_normal((n, k)).astype(np.float32) * 0.02)
    qw = q.FP8Weight(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda())
    x = _bf16(rng, m, k)
    xc, xs = fp8.quantize_rows(x.float().numpy(), fp8.E4M3)
    y = q.qlora_fp8_linear_fwd(qw, x.cuda())
    _check_product(y, fp8.rows_values(xc, xs, fp8.E4M3), fp8.weight_values(codes, scales))
    rows = q.qlora_quantize_fp8_rows(x.cuda())
    assert torch.equal(q.qlora_fp8_linear_fwd(qw, rows), y)          # the same rows, quantized outside
    assert torch.equal(q.qlora_fp8_linear_fwd(qw, x.cuda()), y)      # and again
    assert q.qlora_device_status() == (0, 0)


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("fmt", [0, 1])
def test_backward(q, m, n, k, fmt):
    rng = np.random.default_rng(m * 37 + n + k)
    codes, scales = fp8.quantize_weight(rng.standard_normal((n, k)).astype(np.float32) * 0.02)
    qw = q.FP8Weight(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda())
    dy = _bf16(rng, m, n, scale=1e-3)
    dc, ds = fp8.quantize_rows(dy.float().numpy(), fp8.FORMATS[fmt])
    dx = q.qlora_fp8_linear_bwd(qw, dy.cuda(), fmt=fmt)
    _check_product(dx, fp8.rows_values(dc, ds, fp8.FORMATS[fmt]), fp8.weight_values(codes, scales).T)
    rows = q.qlora_quantize_fp8_rows(dy.cuda(), fmt=fmt)
    assert torch.equal(q.qlora_fp8_linear_bwd(qw, rows), dx)
    assert q.qlora_device_status() == (0, 0)


def test_forward_in_e5m2_rows(q):
    rng = np.random.default_rng(5)
    for m in (3, 40, 300):
        codes, scales = fp8.quantize_weight(rng.standard_normal((500, 528)).astype(np.float32))
        qw = q.FP8Weight(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda())
        x = _bf16(rng, m, 528)
        xc, xs = fp8.quantize_rows(x.float().numpy(), fp8.E5M2)
        y = q.qlora_fp8_linear_fwd(qw, q.qlora_quantize_fp8_rows(x.cuda(), fmt=q.FP8_E5M2))
        _check_product(y, fp8.rows_values(xc, xs, fp8.E5M2), fp8.weight_values(codes, scales))


@pytest.mark.parametrize("m,n,k", [(1, 300, 656), (9, 300, 656), (40, 300, 656), (300, 300, 656), (1300, 2307, 1296)])
def test_scales_of_every_block_count(q, m, n, k):
    # each block with a scale of its own size: a scale taken from a neighbour shows
    rng = np.random.default_rng(m)
    size = np.exp2(rng.integers(-9, 10, (-(-n // 128), -(-k // 128)))).astype(np.float32)
    w = rng.standard_normal((n, k)).astype(np.float32) * np.repeat(np.repeat(size, 128, 0), 128, 1)[:n, :k]
    codes, scales = fp8.quantize_weight(w)
    qw = q.FP8Weight(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda())
    for fwd, cols in ((True, k), (False, n)):
        xs_size = np.exp2(rng.integers(-9, 10, (m, -(-cols // 128))))
        x = (rng.standard_normal((m, cols)) * np.repeat(xs_size, 128, 1)[:, :cols]).astype(np.float32)
        x = torch.from_numpy(x).bfloat16()
        xc, xs = fp8.quantize_rows(x.float().numpy(), fp8.E4M3)
        values, wv = fp8.rows_values(xc, xs, fp8.E4M3), fp8.weight_values(codes, scales)
        if fwd:
            _check_product(q.qlora_fp8_linear_fwd(qw, x.cuda()), values, wv)
        else:
            _check_product(q.qlora_fp8_linear_bwd(qw, x.cuda()), values, wv.T)


@pytest.mark.parametrize("m,n", [(1, 200), (12, 200), (70, 200), (260, 200), (1300, 2307)])
def test_values_that_are_not_finite_stay_in_their_rows(q, m, n):
    rng = np.random.default_rng(m + 1)
    w = q.qlora_quantize_fp8(_bf16(rng, n, 272).cuda())
    x = _bf16(rng, m, 272).cuda()
    y0 = q.qlora_fp8_linear_fwd(w, x)
    x[m // 2, 5] = float("inf")
    y = q.qlora_fp8_linear_fwd(w, x)
    assert torch.all(torch.isnan(y[m // 2]))
    keep = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(y[keep], y0[keep])


def test_rows_of_a_wider_buffer(q):
    # rows further apart than their length, in memory whose other bytes are not codes of theirs
    rng = np.random.default_rng(12)
    w = q.qlora_quantize_fp8(_bf16(rng, 300, 400).cuda())
    for m in (1, 6, 150, 1300):
        x = _bf16(rng, m, 400).cuda()
        rows = q.qlora_quantize_fp8_rows(x)
        wide = torch.full((m, 512), 0x7F, dtype=torch.uint8, device="cuda")
        wide[:, 16:416] = rows.codes.view(torch.uint8)
        shifted = q.FP8Rows(wide.view(torch.float8_e4m3fn)[:, 16:416], rows.scales)
        assert torch.equal(q.qlora_fp8_linear_fwd(w, shifted), q.qlora_fp8_linear_fwd(w, rows))


def test_many_calls_in_flight(q):
    # products, norms and quantizers launched one behind the other, each started before the one in front is
    # done: every result as when called alone
    rng = np.random.default_rng(13)
    w = [q.qlora_quantize_fp8(_bf16(rng, 512, 512, scale=0.05).cuda()) for _ in range(3)]
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    for m in (1, 33, 300, 1500):
        x = _bf16(rng, m, 512).cuda()

        def chain(wait):
            y, out = x, []
            for i in range(9):
                y8, h, _ = q.qlora_rmsnorm_fwd(y, gamma, residual=x, fp8=True)
                y = q.qlora_fp8_linear_fwd(w[i % 3], y8)
                d = q.qlora_fp8_linear_bwd(w[i % 3], y)
                if wait:
                    torch.cuda.synchronize()
                out += [y, h, d]
            return out

        want = chain(True)
        for _ in range(3):
            got = chain(False)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert q.qlora_device_status() == (0, 0)


def test_gradient_is_the_transpose(q):
    # <dY, x W^T> and <dY W, x> over rows that 8 bits hold exactly: y is linear
    # in x, so differences of the forward are the backward's products
    g = torch.Generator().manual_seed(3)
    w = q.qlora_quantize_fp8(torch.randint(-8, 9, (96, 160), generator=g).bfloat16().cuda())
    x = torch.randint(-4, 5, (5, 160), generator=g).bfloat16().cuda()
    x[:, ::128] = 7.0       # scales 7/448: powers of two times integers up to 7 are exact
    dy = torch.randint(-3, 4, (5, 96), generator=g).bfloat16().cuda()
    dy[:, 0] = 3.5
    wf = q.qlora_dequantize_fp8(w).double()
    y = q.qlora_fp8_linear_fwd(w, x).double()
    dx = q.qlora_fp8_linear_bwd(w, dy).double()
    xs, dys = (q.qlora_quantize_fp8_rows(t).dequantize().double() for t in (x, dy))
    a, b = (dys * (xs @ wf.t())).sum(), ((dys @ wf) * xs).sum()
    s = (dys.abs() * (xs.abs() @ wf.abs().t())).sum()
    assert abs(a - b) <= 1e-12 * s
    # each side off by half a bf16 step a value, plus the dequantized weight's own rounding
    assert abs((dys * y).sum() - a) <= 2.0 ** -7 * s and abs((dx * xs).sum() - b) <= 2.0 ** -7 * s


def test_no_rows_outputs_workspaces_and_another_stream(q):
    rng = np.random.default_rng(8)
    w = q.qlora_quantize_fp8(_bf16(rng, 300, 256).cuda())
    assert q.qlora_fp8_linear_fwd(w, torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")).shape == (0, 300)
    assert q.qlora_fp8_linear_bwd(w, torch.empty(0, 300, dtype=torch.bfloat16, device="cuda")).shape == (0, 256)
    x = _bf16(rng, 40, 256).cuda()
    y = q.qlora_fp8_linear_fwd(w, x)
    need = q.qlora_fp8_workspace_bytes(40, 300, 256)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    # only the rows asked for are written
    big = torch.full((50, 300), 9.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(q.qlora_fp8_linear_fwd(w, x, y=big[:40], ws=ws), y) and torch.all(big[40:] == 9.0)
    with pytest.raises(q.QloraError):
        q.qlora_fp8_linear_fwd(w, x, ws=ws[:64])
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(w, x[:, :128])
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(w, x.float())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [q.qlora_fp8_linear_fwd(w, x, stream=side) for _ in range(4)]     # their scratch is the side stream's
    other = [q.qlora_fp8_linear_fwd(w, x) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, y) for t in outs + other)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_captured_and_replayed(q, m):
    rng = np.random.default_rng(m + 2)
    w = q.qlora_quantize_fp8(_bf16(rng, 520, 512).cuda())
    x, dy = _bf16(rng, m, 512).cuda(), _bf16(rng, m, 520).cuda()
    y0, dx0 = q.qlora_fp8_linear_fwd(w, x), q.qlora_fp8_linear_bwd(w, dy)
    graphs = []
    for _ in range(2):       # two graphs, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = q.qlora_fp8_linear_fwd(w, x), q.qlora_fp8_linear_bwd(w, dy)
        graphs.append((g, out))
    x2 = _bf16(rng, m, 512).cuda()
    for data, want in ((x.clone(), y0), (x2, None)):
        x.copy_(data)
        want = q.qlora_fp8_linear_fwd(w, x) if want is None else want
        for g, out in graphs:
            out[0].zero_(), out[1].zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out[0], want) and torch.equal(out[1], dx0)
    assert q.qlora_device_status() == (0, 0)


def test_offsets_past_31_bits(q):
    n, k = 11008, 128
    m = 2 ** 31 // n + 300
    w = q.qlora_quantize_fp8(torch.randn(n, k, device="cuda").bfloat16())
    x = q.qlora_quantize_fp8_rows(torch.randn(m, k, device="cuda").bfloat16())
    y = q.qlora_fp8_linear_fwd(w, x)
    tail = q.FP8Rows(x.codes.view(torch.uint8)[-300:].clone().view(torch.float8_e4m3fn), x.scales[-300:].clone())
    weight = w.codes.float() * w.scales.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    _check_product(y[-300:], tail.dequantize().double().cpu().numpy(), weight.double().cpu().numpy())
