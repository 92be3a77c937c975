"""The oracle of the 8-bit AdamW's states against float64 and against torch's
own arithmetic and casts (no GPU needed)."""

import numpy as np
import torch

from oracle import adamw8, fp8, optim


def test_codes_and_scales_of_a_block():
    rng = np.random.default_rng(4)
    v = np.abs(rng.standard_normal(600)).astype(np.float32)
    v[3], v[4] = 0, 1e-12
    codes, scales = adamw8.encode(v, True)
    assert scales.shape == (3,) and codes[3] == 0 and codes[4] == 1       # above zero stays above zero
    assert adamw8.encode(v, False)[0][4] == 0
    wide = np.repeat(scales.astype(np.float64), 256)[:600]
    # the scale and the inverse are off by two roundings each
    assert np.all(np.abs(scales * 448.0 - [v[:256].max(), v[256:512].max(), v[512:].max()]) <= 2.0 ** -22 * scales * 448)
    off = np.abs(fp8.decode(codes, fp8.E4M3) * wide - v)
    assert np.all(off[5:] <= np.maximum(2.0 ** -4 * v, 2.0 ** -10 * wide)[5:] * (1 + 2.0 ** -18))
    zero = adamw8.encode(np.zeros(5, np.float32), True)
    assert np.all(zero[0] == 0) and zero[1][0] == np.float32(2.0 ** -100) * (np.float32(1) / np.float32(448))


def test_states_against_float64():
    rng = np.random.default_rng(5)
    m, g = (rng.standard_normal(5000).astype(np.float32) for _ in range(2))
    r = np.abs(rng.standard_normal(5000)).astype(np.float32)
    b1, b2 = (float(np.float32(b)) for b in (0.9, 0.999))
    m1, r1 = adamw8.states(m, r, g, b1, b2)
    _, m64, v64 = optim.adamw_step(np.zeros(5000), g, m, r.astype(np.float64) ** 2, 1, 1e-3, b1, b2, 1e-8, 0.0)
    # two roundings of either term of m; v 3, its root 1.5 of them and one of its own
    assert np.all(np.abs(m1 - m64) <= 2.01 * 2.0 ** -24 * (b1 * np.abs(m) + (1 - b1) * np.abs(g)))
    assert np.all(np.abs(r1 - np.sqrt(v64)) <= 2.51 * 2.0 ** -24 * np.sqrt(v64))


def test_a_step_from_torch_operations():
    # the same operations in torch on the CPU, tensors throughout so that each is the one written
    rng = np.random.default_rng(6)
    n = 256 * 40
    own = (np.zeros(n, np.uint8), np.zeros(40, np.float32)) * 2
    one, f, b1, b2 = (torch.tensor(v, dtype=torch.float32) for v in (1.0, 448.0, 0.9, 0.999))
    codes, scales = [torch.zeros(n).to(torch.float8_e4m3fn) for _ in range(2)], [torch.zeros(40) for _ in range(2)]
    for _ in range(3):
        g = torch.from_numpy(rng.standard_normal(n).astype(np.float32))
        own = adamw8.step(*own, g.numpy(), b1.item(), b2.item())
        m, r = (c.float().view(40, 256) * s[:, None] for c, s in zip(codes, scales))
        d = g.view(40, 256)
        m = torch.add(m * b1, d * (one - b1))
        r = torch.sqrt(torch.add((r * r) * b2, (d * d) * (one - b2)))
        for i, v in enumerate((m, r)):
            amax = v.abs().amax(1)
            c = v * (f * (one / amax))[:, None]
            c = torch.where(v > 0, c.clamp_min(2.0 ** -9), c) if i else c
            codes[i], scales[i] = c.clamp(-448, 448).to(torch.float8_e4m3fn).view(-1), amax * (one / f)
        for got, want in zip(own, (codes[0].view(torch.uint8), scales[0], codes[1].view(torch.uint8), scales[1])):
            assert np.array_equal(got, want.numpy())
