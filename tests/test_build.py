"""The build of the library beside its torch binding, with the compilers
replaced by a recorder (no GPU, nothing compiled)."""
import os
import types

import pytest
import torch

import mx_gemm_gb300 as fg
from mx_gemm_gb300 import build


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Records each command and writes its output; .broken: substrings of the commands that fail."""
    rec = types.SimpleNamespace(commands=[], broken=())

    def run(cmd, **kw):
        rec.commands.append(cmd)
        bad = any(b in " ".join(cmd) for b in rec.broken)
        if not bad:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        return types.SimpleNamespace(returncode=int(bad), stdout="", stderr="no such header")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    for name, path in (("OUT", ""), ("LIB", "libfg.so"), ("BINDING", "fg_torch.so"), ("MADE_FOR", "fg_torch.made_for")):
        monkeypatch.setattr(build, name, str(tmp_path / path) if path else str(tmp_path))
    return rec


def test_both_are_built_and_then_up_to_date(compilers):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING) and build.up_to_date()
    n = len(compilers.commands)
    assert build.build() == build.LIB and len(compilers.commands) == n


@pytest.mark.parametrize("broken", ["-c " + os.path.join(build.CSRC, "fg_torch.cpp"), "-ltorch_python"])
def test_the_library_is_built_where_the_binding_cannot_be(compilers, broken):
    compilers.broken = (broken,)
    with open(build.BINDING, "w") as f:
        f.write("of other sources")
    os.utime(build.BINDING, (1, 1))
    with pytest.warns(UserWarning, match="no such header"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and build.library_up_to_date() and not os.path.exists(build.BINDING)
    n = len(compilers.commands)
    with pytest.warns(UserWarning):
        build.build()                                   # the library is not compiled again
    assert not any("nvcc" in c[0] for c in compilers.commands[n:])


def test_a_binding_made_for_another_torch_is_stale(compilers, monkeypatch):
    build.build()
    n = len(compilers.commands)
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    assert build.library_up_to_date() and not build.binding_up_to_date() and not build.up_to_date()
    build.build()                                       # the binding alone
    assert {c[0] for c in compilers.commands[n:]} == {"g++"} and build.up_to_date()


def test_a_binding_made_for_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(fg.moe, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    with pytest.raises(RuntimeError, match="2.0.0.other"):
        fg.moe.binding()
    assert fg.moe.binding_if_built() is None


def test_a_library_that_does_not_compile_is_an_error(compilers):
    compilers.broken = ("fg_decode.cu",)
    with pytest.raises(RuntimeError, match="fg_decode.cu"):
        build.build()


@pytest.fixture
def no_binding(monkeypatch, tmp_path):
    monkeypatch.setattr(fg.moe, "_binding", None)
    monkeypatch.setattr(fg.moe, "BINDING_PATH", str(tmp_path / "fg_torch.so"))


def test_without_the_binding(no_binding):
    """The GEMM's own checks answer; the operators that live in the binding say what is missing."""
    pb = fg.PreshuffledB(fg.BShuf(), torch.zeros(16, dtype=torch.uint8), None)
    with pytest.raises(ValueError, match="CUDA"):
        fg.gemm(torch.zeros(4, 256, dtype=torch.bfloat16), pb)
    with pytest.raises(RuntimeError, match="not built"):
        fg.quantize("mxfp8_b32", torch.zeros(4, 256))


@pytest.mark.gpu
def test_the_gemm_without_the_binding_gives_the_same_bits(monkeypatch, tmp_path):
    a, a_s = fg.quantize("mxfp8_b32", torch.randn(16, 2048, device="cuda"))
    b, b_s = fg.quantize("mxfp8_b32", torch.randn(512, 2048, device="cuda"))
    pb = fg.preshuffle_b("mxfp8_b32", b, b_s)
    want = [fg.gemm(a, pb, a_s, split_k=s) for s in (0, 16)]
    monkeypatch.setattr(fg.moe, "_binding", None)
    monkeypatch.setattr(fg.moe, "BINDING_PATH", str(tmp_path / "fg_torch.so"))
    assert all(torch.equal(fg.gemm(a, pb, a_s, split_k=s), y) for s, y in zip((0, 16), want))
    assert fg.get_error() == fg.FG_OK
