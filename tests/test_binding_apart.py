"""The C library stands without the native part of the Python binding: it is linked and loaded
where torch is missing or the binding is, and only the calls that need the binding say so."""
import os
import subprocess
import sys

import pytest

from dense_blas3_gemm_amd import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


CHECKS = """
assert d.version().startswith("dbgemm ")
assert d.check_args(0, 0, 64, 64, 64, 1.0, 4096, 64, 8192, 64, 0.0, 12288, 64, d.BF16_BF16) == 0
assert d.query_policy(4096, 4096, 4096).startswith("bf16_")
g = object.__new__(d.Gemm)
g.lib, g.device, g.handle, g._stream = d.load_library(), 0, None, 0
for call in (lambda: g.layernorm(None, None), lambda: g.run_act(None, None, None), lambda: g.run_dact(None, None, None, None),
             lambda: g.act_mx(None, None, None, None), lambda: g.act_grad_mx(None, None),
             lambda: g.layernorm_grad(None, None, None, None, None)):
    try:
        call()
    except RuntimeError as e:
        assert WORD in str(e), e
    else:
        raise AssertionError("no error")
"""


def test_library_loads_without_torch():
    run("import sys\nsys.modules['torch'] = None\nimport dense_blas3_gemm_amd as d\nWORD = 'torch'\n" + CHECKS)


def test_library_loads_without_the_binding(tmp_path):
    run(f"import dense_blas3_gemm_amd as d\nd.BINDING_PATH = {str(tmp_path / 'none.so')!r}\nWORD = 'missing'\n" + CHECKS)


def test_library_loads_beside_a_binding_that_does_not(tmp_path):
    bad = tmp_path / "_binding.so"
    bad.write_bytes(b"not a library")
    run(f"import dense_blas3_gemm_amd as d\nd.BINDING_PATH = {str(bad)!r}\nWORD = 'build it again'\n" + CHECKS)


@pytest.fixture
def built(tmp_path, monkeypatch):
    """build() with the compiler and the linker replaced: the output it leaves."""
    out = tmp_path / "lib.so"
    monkeypatch.setattr(b, "OUT", str(out))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "_compile", lambda entry, incremental=False: "x.o")
    monkeypatch.setattr(b, "_write_build_info", lambda: None)

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def link(cmd, **kw):
        if "-o" in cmd and cmd[cmd.index("-o") + 1].startswith(str(out)):
            open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()
    monkeypatch.setattr(b.subprocess, "run", link)
    return out


def test_library_is_linked_where_torch_is_missing(built, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    b.build()
    assert built.exists()


def test_library_is_linked_before_a_binding_that_fails_is_reported(built, monkeypatch):
    def fails(*a, **k):
        raise RuntimeError("g++ failed for binding.cpp")
    monkeypatch.setattr(b, "_build_binding", fails)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        b.build()
    assert built.exists()
