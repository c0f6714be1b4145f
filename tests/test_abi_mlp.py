"""The MLP-block entry points without a GPU: refused without a handle, whatever the sizes."""
import ctypes

import pytest

import dense_blas3_gemm_amd as d

NOT_INITIALIZED = 3


@pytest.mark.parametrize("size", [0, 1, 64])
@pytest.mark.parametrize("name", ["gemm_run_act", "gemm_run_dact", "gemm_act_mx", "gemm_act_grad_mx", "gemm_layernorm",
                                  "gemm_layernorm_grad"])
def test_no_handle(name, size):
    fn = getattr(d.load_library(), name)
    args = [size if t is ctypes.c_int64 else 0.0 if t is ctypes.c_float else 0 if t is ctypes.c_int else None
            for t in fn.argtypes]
    assert fn(*args) == NOT_INITIALIZED
