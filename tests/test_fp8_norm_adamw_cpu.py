"""The oracle of the 8-bit linear and the RMS norm against independent
definitions, and what the library and the binding refuse (no GPU needed:
nothing here launches a kernel)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8, norm


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


TORCH = {"e4m3": (fp8.E4M3, torch.float8_e4m3fn), "e5m2": (fp8.E5M2, torch.float8_e5m2)}


# ---------------------------------------------------------------- oracle pins
@pytest.mark.parametrize("name", ["e4m3", "e5m2"])
def test_fp8_codes_round_trip_and_match_torch(name):
    fmt, dtype = TORCH[name]
    codes = np.arange(256, dtype=np.uint8)
    mine = fp8.decode(codes, fmt)
    theirs = torch.from_numpy(codes).view(dtype).double().numpy()
    assert np.array_equal(mine, theirs, equal_nan=True)
    finite = np.isfinite(mine)
    assert np.array_equal(fp8.encode(mine[finite], fmt), codes[finite])
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(200_000) * np.exp2(rng.uniform(-20, 9, 200_000))).astype(np.float32)
    x = np.clip(x, -fmt["top"], fmt["top"])
    assert np.array_equal(fp8.encode(x, fmt), torch.from_numpy(x).to(dtype).view(torch.uint8).numpy())
    # midpoints go to the even code; beyond the top saturates; NaN is the NaN code
    v = np.unique(mine[finite & (mine >= 0)])
    mid = (v[:-1] + v[1:]) / 2
    assert np.all(fp8.encode(mid, fmt) % 2 == 0)
    assert fp8.decode(fp8.encode([1e30, -1e30], fmt), fmt).tolist() == [fmt["top"], -fmt["top"]]
    assert fp8.encode([np.nan], fmt)[0] == 0x7F


@pytest.mark.parametrize("name", ["e4m3", "e5m2"])
def test_block_quantization_bounds(name):
    fmt, _ = TORCH[name]
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 300)).astype(np.float32)
    x[1] = 0
    x[2, 7] = np.inf
    x[3, 200] = np.nan
    codes, scales = fp8.quantize_rows(x, fmt)
    back = fp8.rows_values(codes, scales, fmt)
    assert scales.shape == (5, 3)
    assert np.all(back[1] == 0) and np.all(np.isfinite(scales))
    bad = ~np.isfinite(x)
    assert np.all(np.isnan(back[bad])) and np.all(np.isfinite(back[~bad]))     # only the value itself is spoiled
    half = 2.0 ** -(fmt["mant"] + 1)
    least = np.repeat(scales, 128, 1)[:, :300] * 2.0 ** (fmt["emin"] - fmt["mant"] - 1)
    off = np.abs(back - x)[~bad]
    assert np.all(off <= np.maximum(half * np.abs(x[~bad]), least[~bad]) * (1 + 1e-5))
    w, sw = fp8.quantize_weight(rng.standard_normal((130, 260)).astype(np.float32))
    assert sw.shape == (2, 3)
    for i, j in ((0, 0), (1, 2)):
        block = fp8.decode(w[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128], fp8.E4M3)
        assert np.abs(block).max() == 448


def test_norm_backward_against_differences():
    rng = np.random.default_rng(2)
    h, gamma, dy = rng.standard_normal((3, 11)), rng.standard_normal(11), rng.standard_normal((3, 11))
    dres, eps = rng.standard_normal((3, 11)), 1e-3

    def loss(h, gamma):
        return np.sum(norm.forward(h, gamma, eps)[0] * dy) + np.sum(h * dres)

    dh, dgamma = norm.backward(dy, h, gamma, norm.forward(h, gamma, eps)[1], dres)
    step = 1e-5
    for grad, which in ((dh, 0), (dgamma, 1)):
        args = [h.copy(), gamma.copy()]
        for i in np.ndindex(grad.shape):
            old = args[which][i]
            args[which][i] = old + step
            up = loss(*args)
            args[which][i] = old - step
            down = loss(*args)
            args[which][i] = old
            assert abs((up - down) / (2 * step) - grad[i]) < 1e-6 * max(1, abs(grad[i]))


# ---------------------------------------------------------------- refusals of the library
def _f(v=16):
    return ctypes.c_void_p(v)


def test_quantizers_refuse(q):
    lib = q.lib
    assert lib.qlora_quantize_fp8(_f(), None, None) == 1
    assert lib.qlora_quantize_fp8(_f(), q.Fp8Struct(4, 24, 16, 16), None) == 2      # K % 16
    assert lib.qlora_quantize_fp8(_f(), q.Fp8Struct(0, 16, 16, 16), None) == 2
    assert lib.qlora_quantize_fp8(_f(), q.Fp8Struct(4, 16, 0, 16), None) == 1
    assert lib.qlora_quantize_fp8(_f(), q.Fp8Struct(4, 16, 24, 16), None) == 3
    assert lib.qlora_quantize_fp8(None, q.Fp8Struct(4, 16, 16, 16), None) == 1
    assert lib.qlora_dequantize_fp8(q.Fp8Struct(4, 16, 16, 16), _f(8), None) == 3
    rows = lambda **k: q.Fp8RowsStruct(*(dict(rows=4, cols=20, ld=32, codes=16, scales=16, format=0, reserved=0) | k).values())  # noqa: E731
    call = lib.qlora_quantize_fp8_rows
    assert call(_f(), None, None) == 1
    assert call(_f(), rows(format=2), None) == 1
    assert call(_f(), rows(reserved=1), None) == 1
    assert call(_f(), rows(ld=16), None) == 2          # rows overlap
    assert call(_f(), rows(ld=40), None) == 2          # not a multiple of 16
    assert call(_f(), rows(cols=0), None) == 2
    assert call(_f(), rows(rows=-1), None) == 2
    assert call(_f(), rows(codes=8), None) == 3
    assert call(_f(), rows(scales=0), None) == 1
    assert call(_f(2), rows(), None) == 3
    assert call(None, rows(rows=0, codes=0, scales=0), None) == 0    # nothing to do


def test_product_refuses(q):
    lib = q.lib
    w = q.Fp8Struct(64, 32, 16, 16)
    x8 = lambda rows=4, cols=32, fmt=0: q.Fp8RowsStruct(rows, cols, 32 if cols <= 32 else 64, 16, 16, fmt, 0)  # noqa: E731
    fwd, bwd = lib.qlora_fp8_linear_fwd, lib.qlora_fp8_linear_bwd
    assert fwd(None, _f(), None, 4, _f(), _f(), 1 << 20, None) == 1
    assert fwd(w, _f(), None, -1, _f(), _f(), 1 << 20, None) == 2
    assert fwd(w, _f(), x8(), 4, _f(), _f(), 1 << 20, None) == 1      # both inputs
    assert fwd(w, None, None, 4, _f(), _f(), 1 << 20, None) == 1      # neither
    assert fwd(w, None, x8(rows=5), 4, _f(), _f(), 1 << 20, None) == 2
    assert fwd(w, None, x8(cols=16), 4, _f(), _f(), 1 << 20, None) == 2
    assert fwd(w, _f(), None, 4, _f(8), _f(), 1 << 20, None) == 3
    assert fwd(w, _f(), None, 0, None, None, 0, None) == 0
    assert bwd(w, _f(), None, 7, 4, _f(), _f(), 1 << 20, None) == 1   # unknown format
    assert bwd(w, None, x8(cols=32), 0, 4, _f(), _f(), 1 << 20, None) == 2   # rows of N are wanted
    assert bwd(w, None, None, 0, 0, None, None, 0, None) == 0
    # rows in 8 bits bring their own format; the argument is ignored
    assert bwd(w, None, x8(rows=0, cols=64), 7, 0, None, None, 0, None) == 0
    assert bwd(w, None, x8(cols=64, fmt=7), 0, 4, _f(), _f(), 1 << 20, None) == 1
    assert q.qlora_fp8_workspace_bytes(0, 64, 32) == 0
    assert q.qlora_fp8_workspace_bytes(4, 64, 24) == 0
    assert q.qlora_fp8_workspace_bytes(4, 64, 32) >= 4 * (64 + 4)


def test_norm_refuses(q):
    fwd, bwd = q.lib.qlora_rmsnorm_fwd, q.lib.qlora_rmsnorm_bwd
    y8 = q.Fp8RowsStruct(4, 64, 64, 16, 16, 0, 0)
    ok = dict(x=16, res=None, g=16, rows=4, d=64, eps=1e-6, h=None, y=16, y8=None, rstd=None)
    f = lambda **k: fwd(*(ok | k).values(), None)  # noqa: E731
    assert f(rows=-1) == 2 and f(d=0) == 2
    assert f(eps=-1.0) == 1 and f(eps=float("nan")) == 1 and f(eps=float("inf")) == 1
    assert f(x=None) == 1 and f(g=None) == 1 and f(y=None) == 1
    assert f(y8=y8) == 1                          # two outputs
    assert f(res=16) == 1 and f(h=16) == 1        # residual and h go together
    assert f(y=None, y8=q.Fp8RowsStruct(4, 32, 64, 16, 16, 0, 0)) == 2
    assert f(x=8) == 3 and f(y=24) == 3
    assert f(rows=0, x=None) == 0
    b = lambda *a: bwd(*a, None)  # noqa: E731
    assert b(16, 16, 16, 16, None, -1, 64, 16, 16, 16, 1 << 20) == 2
    assert b(None, 16, 16, 16, None, 4, 64, 16, 16, 16, 1 << 20) == 1
    assert b(16, 16, 16, None, None, 4, 64, 16, 16, 16, 1 << 20) == 1
    assert b(16, 16, 16, 16, 8, 4, 64, 16, 16, 16, 1 << 20) == 3
    assert b(None, None, None, None, None, 0, 64, None, None, None, 0) == 0
    assert q.qlora_rmsnorm_workspace_bytes(0, 64) == 0 and q.qlora_rmsnorm_workspace_bytes(4, 64) >= 256


def test_adamw_multi_refuses(q):
    lib = q.lib

    def call(rows, bits=32, **h):
        d = np.array(rows, dtype=np.uint64)
        hp = q.AdamwParams(*(dict(lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, step=1) | h).values())
        return lib.qlora_adamw_multi(d.ctypes.data, len(rows), bits, hp, None)

    a = [4096, 0, 8192, 12288, 16384, 0, 0, 16]
    b = [20480, 0, 8192, 24576, 28672, 0, 0, 16]       # the same gradient twice is fine
    assert call([a], bits=16) == 1
    assert call([a], step=0) == 1 and call([a], b1=1.0) == 1 and call([a], eps=0.0) == 1
    assert call([a], lr=float("nan")) == 1 and call([a], lr=float("inf")) == 1 and call([a], wd=float("nan")) == 1
    assert call([[0] + a[1:]]) == 1
    assert call([[4098] + a[1:]]) == 3
    assert call([a], bits=8) == 1                      # no scales
    assert call([a, a]) == 1                           # the same tensor twice
    assert call([a, [4096 + 60] + b[1:]]) == 1         # overlapping masters
    assert call([a, b[:3] + [12288] + b[4:]]) == 1     # the same state twice
    assert call([a, b[:4] + [16384] + b[5:]]) == 1
    assert call([a[:7] + [0]]) == 0                    # nothing to do
    assert lib.qlora_adamw_multi(None, 0, 32, q.AdamwParams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1), None) == 0
    assert lib.qlora_adamw_multi(None, -1, 32, q.AdamwParams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1), None) == 1
    assert lib.qlora_adamw_multi(None, 1, 32, q.AdamwParams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1), None) == 1


# ---------------------------------------------------------------- refusals of the binding
def test_binding_refuses_cpu_tensors_and_bad_handles(q):
    bf, f32, e4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
    z = lambda *s, t=bf: torch.zeros(*s, dtype=torch.uint8 if t is e4 else t).view(t) if t is e4 else torch.zeros(*s, dtype=t)  # noqa: E731
    w = q.FP8Weight(z(4, 32, t=e4), z(1, 1, t=f32))
    for call in (lambda: q.qlora_quantize_fp8(z(4, 32)), lambda: q.qlora_dequantize_fp8(w),
                 lambda: q.qlora_quantize_fp8_rows(z(4, 32)), lambda: q.qlora_fp8_linear_fwd(w, z(2, 32)),
                 lambda: q.qlora_fp8_linear_bwd(w, z(2, 4)), lambda: q.qlora_rmsnorm_fwd(z(2, 32), z(32)),
                 lambda: q.qlora_rmsnorm_bwd(z(2, 32), z(2, 32), z(32), z(2, t=f32)),
                 lambda: q.AdamWGroup([z(8, t=f32)])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        q.FP8Weight(z(4, 32), z(1, 1, t=f32))                       # not 8-bit
    with pytest.raises(ValueError):
        q.FP8Weight(z(4, 32, t=e4).t(), z(1, 1, t=f32))             # not contiguous
    with pytest.raises(ValueError):
        q.FP8Weight(z(4, 32, t=e4), z(2, 1, t=f32))
    with pytest.raises(ValueError):
        q.FP8Rows(z(4, 20, t=e4), z(4, 1, t=f32))                   # rows 20 bytes apart
    with pytest.raises(ValueError):
        q.FP8Rows(z(4, 32, t=e4)[:, ::2], z(4, 1, t=f32))
    with pytest.raises(ValueError):
        q.FP8Rows.empty(4, 32, fmt=2, device="cpu")
    r = q.FP8Rows.empty(4, 20, device="cpu")
    assert r.ld == 32 and r.codes.shape == (4, 20) and r.scales.shape == (4, 1)
    with pytest.raises(ValueError):
        q.AdamWGroup([])
