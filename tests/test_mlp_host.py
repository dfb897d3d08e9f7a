"""Host-side rules of include/lora_mlp.h and its binding, without a GPU."""
import ctypes

import pytest

F = 0x10000        # never dereferenced: the calls below end before the device is touched
OK, NULL, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from deterministic_arithmetic_gb300 import build_lib

    build_lib.build()


def test_packed_backward_of_no_rows_wants_its_gradients():
    """M = 0: da and db, sums over no rows, are written (as zeros), so they have to be there."""
    from deterministic_arithmetic_gb300 import _capi

    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    f = _capi.fn("lora_delta_bwd_packed8", (vp,) * 6 + (ctypes.c_float,) + (i64,) * 4 + (vp,) * 5 + (ctypes.c_size_t, vp))

    def call(da=F, db=F):
        return f(None, None, None, None, None, None, 1.0, 0, 128, 96, 16, None, da, db, None, None, 0, None)

    assert call(da=None) == call(db=None) == NULL
    assert call(da=F + 4) == call(db=F + 8) == ALIGN
