"""The gated and 8-bit integer entry points without a GPU: refused without a handle, and the
binding's reading of their arguments (tensors in host memory are on device -1, a null handle turns
a call whose arguments are in order into NOT_INITIALIZED)."""
import ctypes

import pytest

import dense_blas3_gemm_amd as d

NOT_INITIALIZED = 3


@pytest.mark.parametrize("size", [0, 1, 64])
@pytest.mark.parametrize("name", ["gemm_run_gated", "gemm_run_dgated", "gemm_quantize_i8", "gemm_run_i8",
                                  "gemm_run_gated_i8"])
def test_no_handle(name, size):
    fn = getattr(d.load_library(), name)
    args = [size if t is ctypes.c_int64 else 0.0 if t is ctypes.c_float else 0 if t is ctypes.c_int else None
            for t in fn.argtypes]
    assert fn(*args) == NOT_INITIALIZED


def zeros(*shape, dtype="bfloat16"):
    import torch
    return torch.zeros(*shape, dtype=getattr(torch, dtype))


def run_gated(**kw):
    a = dict(A=zeros(5, 16), Bg=zeros(16, 24), Bu=zeros(16, 24), C=zeros(5, 24), transB=0, alpha=1.0, act="silu",
             bias_g=None, bias_u=None, g=None, u=None)
    assert set(kw) <= set(a)
    return d._load_native().run_gated(0, -1, *{**a, **kw}.values())


def run_dgated(**kw):
    a = dict(A=zeros(5, 16), B=zeros(16, 24), g=zeros(5, 24), u=zeros(5, 24), dg=zeros(5, 24), du=zeros(5, 24),
             transB=0, alpha=1.0, act="silu", h=None, dbias_g=None, dbias_u=None)
    assert set(kw) <= set(a)
    return d._load_native().run_dgated(0, -1, *{**a, **kw}.values())


def quantize_i8(**kw):
    a = dict(src=zeros(5, 24), dst=zeros(5, 24, dtype="int8"), scales=zeros(5, dtype="float32"))
    assert set(kw) <= set(a)
    return d._load_native().quantize_i8(0, -1, *{**a, **kw}.values())


def run_i8(**kw):
    a = dict(A=zeros(5, 16, dtype="int8"), SA=zeros(5, dtype="float32"), B=zeros(16, 24, dtype="int8"),
             SB=zeros(24, dtype="float32"), C=zeros(5, 24), transB=0, act="none", bias=None, residual=None, beta=1.0)
    assert set(kw) <= set(a)
    return d._load_native().run_i8(0, -1, *{**a, **kw}.values())


def run_gated_i8(**kw):
    a = dict(A=zeros(5, 16, dtype="int8"), SA=zeros(5, dtype="float32"), Bg=zeros(16, 24, dtype="int8"),
             SBg=zeros(24, dtype="float32"), Bu=zeros(16, 24, dtype="int8"), SBu=zeros(24, dtype="float32"),
             C=zeros(5, 24), transB=0, act="silu", bias_g=None, bias_u=None, g=None, u=None)
    assert set(kw) <= set(a)
    return d._load_native().run_gated_i8(0, -1, *{**a, **kw}.values())


def test_arguments_in_order():
    f32 = lambda *s: zeros(*s, dtype="float32")  # noqa: E731
    for call in (run_gated, run_dgated, quantize_i8, run_i8, run_gated_i8):
        assert call() == NOT_INITIALIZED
    assert run_gated(Bg=zeros(24, 16), Bu=zeros(24, 16), transB=True, C=f32(5, 24), bias_g=f32(24), bias_u=f32(24),
                     g=zeros(5, 24), u=zeros(5, 24)) == NOT_INITIALIZED
    e4m3 = lambda *s: zeros(*s, dtype="float8_e4m3fn")  # noqa: E731
    assert run_gated(A=e4m3(5, 16), Bg=e4m3(16, 24), Bu=e4m3(16, 24), bias_u=zeros(24)) == NOT_INITIALIZED
    # both weights side by side in one buffer
    w = zeros(16, 48)
    assert run_gated(Bg=w[:, :24], Bu=w[:, 24:]) == NOT_INITIALIZED
    assert run_dgated(dg=f32(5, 24), du=f32(5, 24), h=zeros(5, 24), dbias_g=f32(24), dbias_u=f32(24)) == NOT_INITIALIZED
    assert quantize_i8(src=f32(5, 24)) == NOT_INITIALIZED
    assert run_i8(bias=zeros(24), residual=zeros(5, 24), beta=0.5, C=zeros(5, 24), act="gelu") == NOT_INITIALIZED
    assert run_gated_i8(bias_g=f32(24), bias_u=f32(24), g=zeros(5, 24), u=zeros(5, 24)) == NOT_INITIALIZED


REFUSED = [
    (run_gated, dict(Bu=zeros(16, 23)), "Bu"), (run_gated, dict(Bu=zeros(16, 24, dtype="float32")), "Bu"),
    (run_gated, dict(Bu=None), "Bu"), (run_gated, dict(C=zeros(5, 23)), "op"), (run_gated, dict(A=zeros(5, 15)), "op"),
    (run_gated, dict(transB=1), "op"), (run_gated, dict(act="swish"), "act"),
    (run_gated, dict(bias_g=zeros(23)), "bias_g"), (run_gated, dict(bias_g=zeros(24), bias_u=zeros(24, dtype="float32")), "type"),
    (run_gated, dict(g=zeros(5, 24, dtype="float32")), "g"), (run_gated, dict(u=zeros(24, 5).t()), "row-major"),
    (run_gated, dict(A=zeros(5, 16, dtype="int8"), Bg=zeros(16, 24, dtype="int8"), Bu=zeros(16, 24, dtype="int8")), "bfloat16"),
    (run_dgated, dict(g=None), "g"), (run_dgated, dict(u=zeros(5, 24, dtype="float32")), "u"),
    (run_dgated, dict(du=zeros(5, 24, dtype="float32")), "du"), (run_dgated, dict(dg=zeros(4, 24)), "op"),
    (run_dgated, dict(h=zeros(5, 23)), "h"), (run_dgated, dict(dbias_u=zeros(24)), "dbias_u"),
    (quantize_i8, dict(src=zeros(5, 24, dtype="float16")), "src"), (quantize_i8, dict(dst=zeros(5, 24, dtype="uint8")), "dst"),
    (quantize_i8, dict(scales=zeros(5)), "scales"), (quantize_i8, dict(scales=zeros(4, dtype="float32")), "scales"),
    (quantize_i8, dict(src=zeros(24)), "matrix"),
    (run_i8, dict(A=zeros(5, 16)), "int8"), (run_i8, dict(B=zeros(16, 24, dtype="uint8")), "int8"),
    (run_i8, dict(SA=zeros(24, dtype="float32")), "SA"), (run_i8, dict(SB=None), "SB"),
    (run_i8, dict(C=zeros(5, 24, dtype="int32")), "C"), (run_i8, dict(residual=zeros(5, 24, dtype="float32")), "residual"),
    (run_gated_i8, dict(SBu=zeros(23, dtype="float32")), "SBu"), (run_gated_i8, dict(Bu=zeros(16, 24)), "Bu"),
    (run_gated_i8, dict(bias_u=zeros(25)), "bias_u"),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refused(i):
    call, kw, word = REFUSED[i]
    with pytest.raises(ValueError, match=word):
        call(**kw)


def test_wrong_kinds_of_arguments():
    for call, kw in ((run_gated, dict(alpha="1")), (run_gated, dict(Bu=3)), (run_dgated, dict(u="u")),
                     (run_i8, dict(residual=1.0)), (run_i8, dict(residual=zeros(5, 24), beta=None)),
                     (quantize_i8, dict(scales=2))):
        with pytest.raises(TypeError):
            call(**kw)
