"""Host-side validation of the 4-bit C entry points (no GPU: only calls that
return before any CUDA work)."""

import ctypes

import pytest

import sparse_top_mixture_b200 as stm

A = 16  # an aligned, never followed address
F32, BF16 = stm.DTYPES["f32"], stm.DTYPES["bf16"]


@pytest.mark.parametrize("name", ["moe_mx4_quantize", "moe_mx4_dequantize"])
def test_conversions_validate(name):
    call = getattr(stm.lib(), name)
    for rows, K, dtype in ((-1, 64, BF16), (4, 0, BF16), (4, 48, BF16), (4, -32, BF16), (4, 64, 2), (1 << 31, 32, BF16),
                           (4, 1 << 31, F32)):
        assert call(rows, K, dtype, A, A, A, None) == 1
    for args in ((None, A, A), (A, None, A), (A, A, None), (8, A, A), (A, 24, A), (A, A, 17)):
        assert call(4, 64, BF16, *args, None) == 1
    assert call(0, 64, BF16, None, None, None, None) == 0


def test_permute_rows_validates():
    call = stm.lib().moe_mx4_permute_rows

    def p(**kw):
        return ctypes.byref(stm.Problem(**{**dict(T=64, H=256, E=8, k=2, I=128, dtype="bf16"), **kw}).c())

    assert call(None, A, A, A, A, A, None) == 1
    assert call(p(H=264), A, A, A, A, A, None) == 1  # a multiple of 8, not of 32
    assert call(p(k=9), A, A, A, A, A, None) == 1
    for i in range(5):
        assert call(p(), *[8 if j == i else A for j in range(5)], None) == 1
        assert call(p(), *[None if j == i else A for j in range(5)], None) == 1
    assert call(p(T=0), None, None, None, None, None, None) == 0


BAD_SIZES = [(-1, 4, 64, 64), (4, 0, 64, 64), (4, 257, 64, 64), (4, 4, 0, 64), (4, 4, 64, 0), (4, 4, 64, 48),
             (1 << 31, 4, 64, 64), (4, 4, 1 << 29, 64), (4, 4, 64, 1 << 31), ((1 << 31) - 1, 4, 8192, 64)]


def test_grouped_matmul_validates():
    call = stm.lib().moe_mx4_grouped_matmul
    for sizes in BAD_SIZES + [(4, 4, 60, 64)]:
        assert call(*sizes, BF16, *[A] * 6, None, None) == 1
    assert call(4, 4, 64, 64, 2, *[A] * 6, None, None) == 1
    for i in range(6):
        for bad in (None, 8):
            assert call(4, 4, 64, 64, F32, *[bad if j == i else A for j in range(6)], None, None) == 1
    assert call(4, 4, 64, 64, F32, *[A] * 6, 8, None) == 1  # the workspace
    assert call(0, 4, 64, 64, F32, *[None] * 6, None, None) == 0


def test_grouped_gate_up_validates():
    call = stm.lib().moe_mx4_grouped_gate_up
    for sizes in BAD_SIZES + [(4, 4, 40, 64)]:
        assert call(*sizes, *[A] * 6, None, None, None) == 1
    for i in range(6):
        for bad in (None, 8):
            assert call(4, 4, 64, 64, *[bad if j == i else A for j in range(6)], A, None, None) == 1
    assert call(4, 4, 64, 64, *[A] * 6, 8, None, None) == 1
    assert call(0, 4, 64, 64, *[None] * 6, None, None, None) == 0
