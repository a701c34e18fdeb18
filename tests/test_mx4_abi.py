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


def _tile_table(offsets, BM):
    """csrc/tiles.cuh and the rows that mx4_gemm.cu makes of it, in wrapped 32 bits: (row tiles of each segment, the
    largest row that a lane of any segment's last tile compares with the segment's end)."""
    import numpy as np

    with np.errstate(over="ignore"):
        a, b, m = (np.array(v, dtype=np.int32) for v in (offsets[:-1], offsets[1:], BM))
        counts = (b - a + m - np.int32(1)) // m
        last = a + (counts - np.int32(1)) * m + m - np.int32(1)
    return counts.tolist(), last.tolist()


def _statuses_without_a_device(sizes):
    """Of both products for each (rows, K), in a process that sees no GPU: 1 where the sizes are refused, another error
    (no device) where they are accepted. Nothing can be launched there."""
    import os
    import subprocess
    import sys

    code = (f"import sparse_top_mixture_b200 as stm; L = stm.lib(); A = 16\n"
            f"for rows, K in {sizes}:\n"
            f"    print(L.moe_mx4_grouped_matmul(rows, 1, 8, K, 1, *[A] * 6, None, None),"
            f" L.moe_mx4_grouped_gate_up(rows, 1, 32, K, *[A] * 6, None, None, None))")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}, cwd=root,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return [[int(v) for v in line.split()] for line in r.stdout.splitlines()]


def test_rows_next_to_32_bits():
    """Where rows or tiles would wrap, the products refuse; the largest accepted count wraps nowhere."""
    shorts = [0, 1, 127, 128, 255, 256]
    statuses = _statuses_without_a_device([((1 << 31) - 1 - short, 32) for short in shorts])
    for short, status in zip(shorts, statuses):
        rows = (1 << 31) - 1 - short
        wraps = False
        for offsets in ([0, rows], [0, 1, rows], [0, rows - 1, rows]):
            for BM in (128, 256):
                counts, last = _tile_table(offsets, BM)
                wraps |= any(c != -(-(b - a) // BM) for a, b, c in zip(offsets, offsets[1:], counts))
                wraps |= any(b > a and row < b - 1 for a, b, row in zip(offsets, offsets[1:], last))
        assert wraps == (short < 255)
        assert (status == [1, 1]) == (short < 256)


def test_rows_too_long_for_the_bounded_waits():
    """A K of 2^27 or more, whose tiles could outlast a wait, is refused."""
    assert _statuses_without_a_device([(4, 1 << 27)]) == [[1, 1]]
    assert all(s not in (0, 1) for s in _statuses_without_a_device([(4, (1 << 27) - 32)])[0])
