"""Host argument checks (no GPU) of the gradient calls: buffers that one part of a
call would write while another reads them are refused before anything is launched."""
import ctypes

import pytest

from helpers import ensure_built

P, MB = 1 << 30, 1 << 20


@pytest.fixture(scope="module")
def L():
    ensure_built()
    import boolean_weight_matmul_b200 as mb
    return mb.lib()


def test_scale_gradients_refuse_the_buffers_they_are_computed_from(L):
    import torch
    arr = lambda *v: ctypes.cast((ctypes.c_void_p * len(v))(*v), ctypes.c_void_p)
    ia = lambda *v: ctypes.cast((ctypes.c_int * len(v))(*v), ctypes.c_void_p)
    # two matrices of 64 and 40 rows, N = 1024, 40 tokens: X and dX 81920 bytes, dY 5120 and 3200, dalpha 6144 and 2560
    call = lambda X, dY, dX, da: L.mbok_gemm_backward(2, arr(P, P), arr(P, P), ia(3, 2), ia(64, 40), 1024, 128, X, 40,
                                                      arr(*dY), dX, arr(*da), P, 1 << 26, None)
    x, dy0, dy1, dx, da0, da1 = (P + (i + 1) * MB for i in range(6))
    for bad in (x, x + 81904, x - 6128, dy0 + 5104, dy0 - 6128, dy1, dy1 + 3184, dx, dx + 81904, dx - 6128):
        assert call(x, (dy0, dy1), dx, (bad, da1)) == 1
    for bad in (x - 2544, dy0 - 2544, dy1 + 3184, dx - 2544):
        assert call(x, (dy0, dy1), dx, (None, bad)) == 1 and call(x, (dy0, dy1), dx, (da0, bad)) == 1
    assert call(x, (dy0, dy1), None, (x, da1)) == 1             # also without dX
    assert call(x, (dy0, dy1), None, (dy1, None)) == 1
    if not torch.cuda.is_available():                           # buffers that touch reach the launch, which fails here
        for good in (x + 81920, x - 6144, dy0 + 5120, dy1 + 3200, dx + 81920, dx - 6144):
            assert call(x, (dy0, dy1), dx, (good, da1)) == 5
        assert call(x, (dy0, dy1), dx, (None, dy1 - 2560)) == 5
