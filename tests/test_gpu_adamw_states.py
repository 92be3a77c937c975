"""The 8-bit AdamW's states over several steps, bit for bit with an oracle that
keeps states of its own: nothing of the kernel's enters the expectation."""

import numpy as np
import pytest
import torch

from oracle import adamw8, optim

pytestmark = pytest.mark.gpu
HP = dict(lr=2e-3, betas=(0.9, 0.995), eps=1e-8, weight_decay=0.01)
LR, B1, B2, EPS, WD = (float(np.float32(v)) for v in (2e-3, 0.9, 0.995, 1e-8, 0.01))
SIZES = [1, 7, 255, 256, 257, 2048, 4097, 0, 70001, 400_000]


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


def _states(rng, n):
    """Codes and scales as steps leave them: a block's largest code is 448, roots are not negative."""
    nb = -(-n // 256)
    m = rng.standard_normal(n).astype(np.float32) * np.exp2(rng.uniform(-9, 0, n)).astype(np.float32)
    r = np.abs(rng.standard_normal(n)).astype(np.float32)
    size = np.repeat(np.exp2(rng.uniform(-14, -4, nb)).astype(np.float32), 256)[:n]
    return adamw8.encode(m * size, False) + adamw8.encode(r * size, True)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("fresh", [False, True])
def test_states_over_steps_bit_for_bit(q, offset, fresh):
    rng = np.random.default_rng(11 + offset)
    masters = [torch.from_numpy(rng.standard_normal(n + offset).astype(np.float32) * 0.02).cuda()[offset:] for n in SIZES]
    own = [(np.zeros(n, np.uint8), np.zeros(-(-n // 256), np.float32)) * 2 if fresh else _states(rng, n) for n in SIZES]
    group = q.AdamWGroup(masters, bits=8)
    starts = np.concatenate([[0], np.cumsum([-(-n // 256) * 256 for n in SIZES])]).astype(int)
    parts = (group.m.view(torch.uint8), group.m_scales, group.v.view(torch.uint8), group.v_scales)
    cut = [[t[a:a + n] if t.dtype is torch.uint8 else t[a // 256:a // 256 + -(-n // 256)] for t in parts]
           for a, n in zip(starts, SIZES)]
    for views, state in zip(cut, own):
        for t, s in zip(views, state):
            t.copy_(torch.from_numpy(s))
    for t in range(1, 4):
        grads = [rng.standard_normal(n + offset).astype(np.float32) * np.float32(0.01) for n in SIZES]
        for g in grads:
            g[100:150] *= np.float32(1e-6)          # values far below their block's largest
            g[-2:] = 0
        before = [p.double().cpu().numpy() for p in masters]
        q.qlora_adamw_multi(group, [torch.from_numpy(g).cuda()[offset:] for g in grads], t, **HP)
        torch.cuda.synchronize()
        for i, n in enumerate(SIZES):
            if n == 0:
                continue
            g = grads[i][offset:]
            m, r = adamw8.decode(*own[i][:2]), adamw8.decode(*own[i][2:])
            own[i] = adamw8.step(*own[i], g, B1, B2)
            for name, got, want in zip(("m", "m_scales", "v", "v_scales"), cut[i], own[i]):
                got = got.cpu().numpy()
                assert np.array_equal(got, want), (name, n, t, int(np.sum(got != want)))
            # the master from the same states, in roundings of 2^-24: p, its decay factor and the sum one each;
            # of the update, with m's terms by their magnitudes since they may cancel: m two, the root 2.5, its
            # correction and eps two, the reciprocal two (its last bit), the quotient, the step size and the
            # sum one each: under 12, and 16 with the terms of higher order
            new = optim.adamw_step(before[i], g.astype(np.float64), m, r.astype(np.float64) ** 2, t, LR, B1, B2, EPS, WD)
            up = LR / (1 - B1 ** t) / (np.sqrt(new[2]) / np.sqrt(1 - B2 ** t) + EPS)
            size = B1 * np.abs(m).astype(np.float64) + (1 - B1) * np.abs(g).astype(np.float64)
            tol = 2.0 ** -24 * (3 * np.abs(before[i]) + 16 * up * size)
            assert np.all(np.abs(masters[i].double().cpu().numpy() - new[0]) <= tol)
    assert q.qlora_device_status() == (0, 0)


def test_the_same_from_torch_operations(q):
    # the definition as a program of elementary operations states it: amax / 448 and 448 / amax are products
    # with a reciprocal, on either side
    n = 1 << 20
    g = torch.Generator(device="cuda").manual_seed(3)
    group = q.AdamWGroup([torch.zeros(n, device="cuda")], bits=8)
    codes = [torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    scales = [torch.zeros(n // 256, device="cuda") for _ in range(2)]
    for t in (1, 2, 3):
        grad = torch.randn(n, generator=g, device="cuda") * 1e-3
        q.qlora_adamw_multi(group, [grad], t, betas=(0.9, 0.999))
        m, r = (c.float().view(-1, 256) * s[:, None] for c, s in zip(codes, scales))
        b1, b2 = (float(np.float32(b)) for b in (0.9, 0.999))
        d = grad.view(-1, 256)
        m = m * b1 + d * (1 - b1)
        r = torch.sqrt((r * r) * b2 + (d * d) * (1 - b2))
        for i, v in enumerate((m, r)):
            amax = v.abs().amax(1).clamp_min(2.0 ** -100)
            c = (v * (amax.reciprocal() * 448)[:, None]).clamp(-448, 448)
            codes[i] = (torch.where(v > 0, c.clamp_min(2.0 ** -9), c) if i else c).to(torch.float8_e4m3fn).view(-1)
            scales[i] = amax * float(np.float32(1) / np.float32(448))
        for got, want in zip((group.m, group.v), codes):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
        assert torch.equal(group.m_scales, scales[0]) and torch.equal(group.v_scales, scales[1])

