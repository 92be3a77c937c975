"""The 8-bit AdamW step with an eps that a reciprocal has no normal number for:
as the 32-bit step, whose quotient is a division."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.1e-38, 1e-8, 3e38])
@pytest.mark.parametrize("offset", [0, 1])
def test_first_step_as_with_32_bit_states(q, eps, offset):
    n = 4096 + 77
    g = torch.Generator().manual_seed(1)
    p = torch.randn(n + offset, generator=g).cuda()[offset:]
    grad = torch.randn(n + offset, generator=g)
    grad[:400] = 0                           # nothing but eps in the denominator, and nothing above it
    grad[400:500] *= 1e-24                   # squares that fp32 holds as zero, above it m alone
    grad = grad.cuda()[offset:]
    outs, lr = [], 1e-4
    for bits in (8, 32):
        master, copy = p.clone(), p.bfloat16()
        group = q.AdamWGroup([master], params=[copy], bits=bits)
        q.qlora_adamw_multi(group, [grad], 1, lr=lr, eps=eps, weight_decay=0.01)
        assert torch.equal(copy, master.bfloat16())
        outs.append(master.double())
    eight, full = outs
    assert torch.all(torch.isfinite(full)) and torch.all(torch.isfinite(eight))
    zero = grad == 0
    assert torch.equal(eight[zero], full[zero])
    # both from zero states: m = (1 - b1) g alike; the roots, the quotients and the two sums round apart, each
    # under eight roundings of the update and one of the result
    step = (full - p.double() * float(np.float32(1 - float(np.float32(lr)) * float(np.float32(0.01))))).abs()
    assert torch.all((eight - full).abs() <= 2.0 ** -24 * (16 * step + 2 * full.abs() + 2 * p.double().abs()))
    assert q.qlora_device_status() == (0, 0)
