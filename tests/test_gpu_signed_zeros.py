"""Codes of zeros and of values that round to zero keep their sign, in every
quantizer alike: fp8(clamp(v inv)) of the block quantization, bit for bit."""

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


def _values(rows, cols):
    rng = np.random.default_rng(rows + cols)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x[:, ::5] = -0.0
    x[:, 1::5] = 0.0
    x[:, 2::5] *= np.float32(1e-9)        # codes of zero, of either sign
    x[0, :min(cols, 100)] = -0.0
    x[-1, 3] = np.nan
    return torch.from_numpy(x).bfloat16()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows,cols", [(3, 264), (5, 131), (2, 20000), (300, 1024)])
def test_rows(q, fmt, rows, cols):
    x = _values(rows, cols)
    got = q.qlora_quantize_fp8_rows(x.cuda(), fmt=fmt)
    codes, scales = fp8.quantize_rows(x.float().numpy(), fp8.FORMATS[fmt])
    assert np.array_equal(got.codes.contiguous().view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(got.scales.cpu().numpy(), scales)
    assert np.any(codes == 0x80) and np.any(codes == 0)


@pytest.mark.parametrize("n,k", [(3, 272), (300, 512)])
def test_weight(q, n, k):
    w = _values(n, k)
    got = q.qlora_quantize_fp8(w.cuda())
    codes, scales = fp8.quantize_weight(w.float().numpy())
    assert np.array_equal(got.codes.view(torch.uint8).cpu().numpy(), codes)
    assert np.any(codes == 0x80) and np.any(codes == 0)


def test_norm(q):
    x = _values(4, 256)[:3]
    gamma = torch.ones(256, dtype=torch.bfloat16)
    y, _, _ = q.qlora_rmsnorm_fwd(x.cuda(), gamma.cuda(), fp8=True)
    codes = y.codes.view(torch.uint8).cpu()
    assert torch.equal(codes >= 128, torch.signbit(x))
    assert torch.all((codes & 127)[x == 0] == 0)
