"""The native binding's reading of arguments, without a GPU: tensors in host memory are on device
-1, and a null handle turns a call whose arguments are in order into NOT_INITIALIZED."""
import pytest

import dense_blas3_gemm_amd as d

NOT_INITIALIZED = 3


def run_act(z=None, z_scales=None, transA=0, transB=0, alpha=1.0, beta=1.0, residual=None):
    import torch
    A, B, C = (torch.zeros(32, 32, dtype=torch.bfloat16) for _ in range(3))
    return d._load_native().run_act(0, -1, A, B, C, transA, transB, alpha, "relu", None, residual, beta, z, z_scales)


def test_arguments_in_order():
    import torch
    q, s = torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(32, 1, dtype=torch.uint8)
    z = torch.zeros(32, 32, dtype=torch.bfloat16)
    assert run_act() == run_act(z=z) == run_act(z=q, z_scales=s) == run_act(transA=True, transB=1) == NOT_INITIALIZED


def test_scales_without_codes_are_refused():
    """(the checkpoint would not be written)"""
    import torch
    with pytest.raises(ValueError, match="z"):
        run_act(z_scales=torch.zeros(32, 1, dtype=torch.uint8))


@pytest.mark.parametrize("name", ["transA", "transB"])
def test_a_flag_without_a_truth_value(name):
    import torch
    for bad in (torch.zeros(2), object):
        if bad is object:
            class Neither:
                def __bool__(self):
                    raise RuntimeError("neither")
            bad = Neither()
        with pytest.raises(TypeError, match="flag"):
            run_act(**{name: bad})


def test_numbers():
    for kw in (dict(alpha="1"), dict(alpha=None)):
        with pytest.raises(TypeError, match="number"):
            run_act(**kw)
