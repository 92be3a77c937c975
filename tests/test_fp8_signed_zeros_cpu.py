"""The oracle's block quantization against torch's casts, signs of zeros
included (no GPU needed)."""

import numpy as np
import pytest
import torch

from oracle import fp8


@pytest.mark.parametrize("fmt,dtype", [(0, torch.float8_e4m3fn), (1, torch.float8_e5m2)])
def test_codes_of_zeros_keep_their_sign(fmt, dtype):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 200)).astype(np.float32)
    x[:, ::3] = -0.0
    x[:, 1::3] *= np.float32(1e-9)
    f = fp8.FORMATS[fmt]
    codes, _ = fp8.quantize_rows(x, f)
    for block in (slice(0, 128), slice(128, 200)):
        amax = np.abs(x[:, block]).max(1, keepdims=True)
        v = torch.from_numpy(x[:, block] * (np.float32(f["top"]) / amax)).clamp(-f["top"], f["top"])
        assert np.array_equal(codes[:, block], v.to(dtype).view(torch.uint8).numpy())
    assert np.array_equal(codes >= 128, np.signbit(x))
