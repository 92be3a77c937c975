"""Sizes at the limits of the 8-bit product (no GPU needed: nothing launches)."""

import ctypes

import pytest

SHAPE = 2
MOST = 1 << 30          # columns are 32-bit numbers in the kernels


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


def test_reductions_past_the_limit_are_refused_in_bf16_as_in_8_bits(q):
    at = ctypes.c_void_p(16)
    ws = 1 << 50                                # "enough": the sizes are what is refused
    for m in (0, 1, 8):
        wide = q.Fp8Struct(16, MOST + 16, 16, 16)
        assert q.lib.qlora_fp8_linear_fwd(wide, at, None, m, at, at, ws, None) == SHAPE
        # dX reduces over the outputs; 2^31 - 1 of them overflowed the rows' quantizer, which then wrote nothing
        for n in (MOST + 1, (1 << 31) - 4096, (1 << 31) - 1):
            tall = q.Fp8Struct(n, 16, 16, 16)
            assert q.lib.qlora_fp8_linear_bwd(tall, at, None, 0, m, at, at, ws, None) == SHAPE
            rows = q.Fp8RowsStruct(m, n, (n + 15) // 16 * 16, 16, 16, 0, 0)
            assert q.lib.qlora_fp8_linear_bwd(tall, None, rows, 0, m, at, at, ws, None) == SHAPE
    # as many outputs as that are no reduction of the forward
    assert q.lib.qlora_fp8_linear_fwd(q.Fp8Struct(MOST + 1, 16, 16, 16), at, None, 0, at, None, 0, None) == 0
    assert q.lib.qlora_fp8_linear_bwd(q.Fp8Struct(MOST, 16, 16, 16), at, None, 0, 0, at, None, 0, None) == 0
