"""The 8-bit linear, the RMS norm and the many-tensor AdamW together, as a
training step of a pre-norm block uses them: norm -> rows in 8 bits -> frozen
8-bit projection (a merged weight) and an adapted NF4 projection on the same
normed input; gradients back to the residual stream, the norm's gain and the
adapters; one optimizer call over all of them."""

import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


def _rel(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("m", [1, 300])
def test_training_step_of_a_block(q, m):
    k, n, r, alpha, eps = 512, 640, 8, 16.0, 1e-5
    g = torch.Generator().manual_seed(m)
    x, res = (torch.randn(m, k, generator=g).bfloat16().cuda() for _ in range(2))
    gamma32 = (1 + 0.1 * torch.randn(k, generator=g)).cuda()
    gamma = gamma32.bfloat16()
    a32, b32 = synth.lora_a(r, k, seed=1).float().cuda(), synth.lora_b(n, r, seed=1).float().cuda()
    a, b = a32.bfloat16(), b32.bfloat16()
    qw = q.qlora_quantize_nf4(synth.weight(n, k, seed=2).cuda())
    # a second projection whose adapters were merged, kept in 8 bits
    w8 = q.qlora_quantize_fp8(q.qlora_merge_lora(q.qlora_quantize_nf4(synth.weight(n, k, seed=3).cuda()), a, b, alpha))
    group = q.AdamWGroup([a32, b32, gamma32], params=[a, b, gamma], bits=8)
    dy1, dy2 = (torch.randn(m, n, generator=g).mul(0.01).bfloat16().cuda() for _ in range(2))
    dh = torch.randn(m, k, generator=g).mul(0.01).bfloat16().cuda()

    w_hat, w8_hat = q.qlora_dequantize(qw).double(), w8.codes.double() * w8.scales.double().repeat_interleave(128, 0)[
        :n].repeat_interleave(128, 1)[:, :k]
    for step in (1, 2):
        y8, h, rstd = q.qlora_rmsnorm_fwd(x, gamma, eps, residual=res, fp8=True)
        yb, _, _ = q.qlora_rmsnorm_fwd(h, gamma, eps)
        out8 = q.qlora_fp8_linear_fwd(w8, y8)
        out4, u = q.qlora_linear_fwd(qw, yb, a, b, alpha)
        d8 = q.qlora_fp8_linear_bwd(w8, dy1, fmt=q.FP8_E5M2)
        d4, da, db = q.qlora_linear_bwd(qw, yb, u, dy2, a, b, alpha)
        dx, dgamma = q.qlora_rmsnorm_bwd((d8.float() + d4.float()).bfloat16(), h, gamma, rstd, dres=dh)

        # the same in float64 with autograd
        hd = (x.float() + res.float()).bfloat16().double().requires_grad_()
        ad, bd, gd = (t.double().requires_grad_() for t in (a, b, gamma))
        yd = hd * (hd.square().mean(1, keepdim=True) + eps).rsqrt() * gd
        o8, o4 = yd @ w8_hat.t(), yd @ w_hat.t() + alpha / r * (yd @ ad.t()) @ bd.t()
        ((o8 * dy1.double()).sum() + (o4 * dy2.double()).sum() + (hd * dh.double()).sum()).backward()
        # rows in e4m3 (half step 2^-4, uniform: 2^-4 / sqrt(3) of a value at most) and gradients in e5m2 (2^-3)
        assert _rel(out8, o8) <= 2.0 ** -4 / 3 ** 0.5 + 2.0 ** -8
        assert _rel(out4, o4) <= 1e-2
        # the 8-bit path's share of the gradient carries at most 2^-3 / sqrt(3)
        assert _rel(dx, hd.grad) <= 2.0 ** -3 / 3 ** 0.5 + 1e-2
        assert _rel(dgamma, gd.grad) <= 2.0 ** -3 / 3 ** 0.5 + 1e-2
        assert _rel(da, ad.grad) <= 1e-2 and _rel(db, bd.grad) <= 1e-2
        before = [t.clone() for t in (a32, b32, gamma32)]
        q.qlora_adamw_multi(group, [da, db, dgamma], step, lr=1e-3)
        for t, o, copy in zip((a32, b32, gamma32), before, (a, b, gamma)):
            # after two steps |m| / sqrt(v), bias-corrected, is at most 1.002, and at most 2.2 where a code of m
            # was rounded up to twice its value and one of sqrt(v) down to two thirds
            assert not torch.equal(t, o) and float((t - o).abs().max()) <= 2.2e-3 and torch.equal(copy, t.bfloat16())
    assert q.qlora_device_status() == (0, 0)


def test_norm_rows_feed_the_product_as_its_own_quantizer_does(q):
    # 8-bit rows straight from the norm against quantizing the fp32 values of the same rows: the
    # codes come from y before its rounding to bf16, so they may differ by that rounding only
    g = torch.Generator().manual_seed(9)
    x = torch.randn(70, 528, generator=g).bfloat16().cuda()
    gamma = torch.ones(528, dtype=torch.bfloat16, device="cuda")
    w = q.qlora_quantize_fp8(torch.randn(200, 528, generator=g).mul(0.05).bfloat16().cuda())
    y8, _, _ = q.qlora_rmsnorm_fwd(x, gamma, fp8=True)
    yb, _, _ = q.qlora_rmsnorm_fwd(x, gamma)
    assert _rel(y8.dequantize(), yb) <= 2.0 ** -4 / 3 ** 0.5 + 2.0 ** -8
    assert _rel(q.qlora_fp8_linear_fwd(w, y8), q.qlora_fp8_linear_fwd(w, yb)) <= 2.0 ** -4
