"""Which sizes of the block-scaled products are refused: output tiles are numbered with 32
bits.  All on the host: a call that passes the check of sizes is stopped by its NULL output."""
from __future__ import annotations

import pytest

BAD = 0x1000  # never dereferenced


def dense(L, m, n, tiles=False):
    return L.fp8_gemm_block(BAD, 0, BAD, BAD, 0, BAD, 0, 1 if tiles else 128, m, n, 128, None, 1, 0, None)


def grouped(L, groups, rows, n, layout=0):
    return L.fp8_gemm_block_grouped(groups, BAD, BAD, 0, BAD, BAD, 0, BAD, layout, rows, n, 128, None, 0, None)


def wgrad(L, groups, m, n):
    return L.fp8_gemm_block_grouped_wgrad(groups, BAD, BAD, 0, BAD, BAD, 0, BAD, m, n, 128, None, 1, 0, None)


@pytest.mark.parametrize("call", [
    lambda L: grouped(L, 1024, 524288, 16384),         # 4.3e6 tiles of 16 x 128
    lambda L: grouped(L, 1024, 524288, 16384, 1),
    lambda L: grouped(L, 1024, 2 ** 24, 2 ** 13),      # 6.7e7
    lambda L: grouped(L, 2, 2 ** 20, 2 ** 17),
    lambda L: wgrad(L, 1024, 2 ** 17, 2 ** 9),
    lambda L: wgrad(L, 256, 18432, 7168),
    lambda L: wgrad(L, 1024, 1, 2 ** 27),              # 2^29 tiles of 256 columns
    lambda L: dense(L, 2 ** 20, 2 ** 17),
    lambda L: dense(L, 2 ** 18, 2 ** 19, True),
    lambda L: dense(L, 1, 2 ** 31 - 256),
    lambda L: dense(L, 2 ** 31 - 256, 1),
])
def test_calls_that_fit_the_memory_are_not_too_many_tiles(native_lib, call):
    assert call(native_lib) == 1
    assert "d is NULL" in native_lib.fp8_last_error_message().decode()


@pytest.mark.parametrize("call", [
    lambda L: dense(L, 2 ** 21, 2 ** 21),              # 2^31 tiles of 16 x 128
    lambda L: dense(L, 2 ** 21, 2 ** 21, True),
    lambda L: grouped(L, 8, 2 ** 21, 2 ** 21),
    lambda L: grouped(L, 1024, 2 ** 30, 2 ** 14),
    lambda L: wgrad(L, 1024, 2 ** 19, 2 ** 19),
])
def test_calls_whose_tiles_have_no_numbers_are_refused(native_lib, call):
    assert call(native_lib) == 2
    assert "too many output tiles" in native_lib.fp8_last_error_message().decode()
