"""Scratch of the block-scaled linear's backward, by the gradients that are asked for (no GPU)."""
import itertools

import pytest

from test_fp8_refusals import INVALID, WORKSPACE, lib, mem  # noqa: F401  (fixtures)

ERROR_BLOCK = 256


@pytest.mark.parametrize("rows,K,N", [(1, 16, 16), (70, 272, 176), (1003, 1296, 2064), (8192, 4096, 14336)])
def test_bytes(lib, rows, K, N):
    of = lambda *need: lib.dg_fp8_linear_bwd_workspace_bytes_for(rows, K, N, *need)
    every = lib.dg_fp8_linear_bwd_workspace_bytes(rows, K, N)
    assert of(1, 1, 1) == every and of(0, 0, 0) == ERROR_BLOCK
    up = lambda n: -(-n // 256) * 256
    # the weight's gradient needs x in bf16, the input's dy in 8 bits and (from 2048 rows) the weight's codes
    assert of(0, 1, 0) == ERROR_BLOCK + up(2 * rows * K)
    turned = N * K if rows >= 2048 else 0
    assert of(1, 0, 0) == ERROR_BLOCK + up(rows * N) + up(rows * -(-N // 128)) + up(turned)
    assert ERROR_BLOCK < of(0, 0, 1) <= ERROR_BLOCK + up(4 * N * 1216)
    scratch = {n: of(*n) - ERROR_BLOCK for n in itertools.product((0, 1), repeat=3)}
    for n, size in scratch.items():
        assert size == sum(scratch[tuple(int(i == j) for j in range(3))] for i in range(3) if n[i])


def test_refusals(lib, mem):
    assert lib.dg_fp8_linear_bwd_workspace_bytes_for(2, 100, 16, 1, 1, 1) == 0
    xc, xs, wc, ws, dy, dx, dw, db, w = mem[:9]

    def call(dx, dw, db, n):
        return lib.dg_fp8_linear_bwd(2, 128, 16, xc, xs, wc, ws, dy, dx, dw, db, w, n, None)

    for out in ((dx, None, None), (None, dw, None), (None, None, db), (dx, None, db), (dx, dw, db)):
        need = lib.dg_fp8_linear_bwd_workspace_bytes_for(2, 128, 16, *(int(t is not None) for t in out))
        assert call(*out, need - 1) == WORKSPACE
    # an output may lie where the workspace ends for the gradients asked for, and not before
    at = w + lib.dg_fp8_linear_bwd_workspace_bytes_for(2, 128, 16, 1, 0, 0)
    assert call(at - 256, None, None, 1 << 16) == INVALID and b"overlaps" in lib.dg_last_error()
