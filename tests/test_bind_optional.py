"""Only the 4-bit and expert-layer calls need _tb_bind.so: without it, or with
one built for another torch, the library and every other call still load and
build, and those calls raise with the reason."""
import os
import subprocess
import sys

import pytest
import torch

from decode_gemv_tb_b200 import build as tbbuild
from decode_gemv_tb_b200 import tb

NAME = "decode_gemv_tb_b200._tb_bind"


@pytest.fixture
def unloaded(monkeypatch):
    tbbuild.build()
    monkeypatch.setattr(tb, "_lib", None)
    monkeypatch.setattr(tb, "_bind", None)


def refused(what):
    u8 = torch.zeros(512, dtype=torch.uint8)
    w, x = torch.zeros(4, 64), torch.zeros((2, 128), dtype=torch.bfloat16)
    for call in (lambda: tb.tb_mx4_quantize(w), lambda: tb.tb_mx4_dequantize(u8, u8, 4, 64),
                 lambda: tb.tb_mx4_gemm(u8, u8, u8, u8, 2, 4, 64), lambda: tb.tb_moe_route(x, x, 1)):
        with pytest.raises(tb.TBError, match=what):
            call()


def test_scalar_calls_load_without_it(unloaded, monkeypatch):
    monkeypatch.setitem(sys.modules, NAME, None)  # its import fails
    assert tb.load().tb_version() >= 100
    assert tb.packed_bytes(tb.INT2, 4, 128) == 128 and tb.mx4_code_bytes(4, 64) == 128
    refused("_tb_bind.so: .*run `python -m")


def test_another_torch_is_told(unloaded, monkeypatch):
    class Other:
        built_for = "torch 0.1, python 3.12"

        @staticmethod
        def init(*_):
            raise AssertionError("a call into a module built for another torch")

    monkeypatch.setitem(sys.modules, NAME, Other)
    assert tb.load().tb_version() >= 100
    refused("built for torch 0.1")


def compiler(tmp_path, name, text):
    """A compiler that writes `text` to the file behind -o."""
    p = tmp_path / name
    p.write_text(f"""#!/bin/sh
while [ $# -gt 1 ]; do
    if [ "$1" = -o ]; then printf '{text}' > "$2"; fi
    shift
done
""")
    p.chmod(0o755)
    return str(p)


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    monkeypatch.setattr(tbbuild, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(tbbuild, "BIND", str(tmp_path / "bind.so"))
    monkeypatch.setattr(tbbuild, "NVCC", compiler(tmp_path, "nvcc", "library"))
    return tmp_path


@pytest.mark.parametrize("left_over", [False, True])
def test_builds_the_library_without_a_host_compiler(elsewhere, monkeypatch, left_over):
    monkeypatch.setenv("CXX", str(elsewhere / "no_such_compiler"))
    if left_over:
        (elsewhere / "bind.so").write_text("of an older tb.h")
        os.utime(elsewhere / "bind.so", (1, 1))
    with pytest.warns(UserWarning, match="_tb_bind.so not built"):
        tbbuild.build()
    assert (elsewhere / "lib.so").read_text() == "library"
    assert not (elsewhere / "bind.so").exists()  # nothing that no longer fits stays
    with pytest.raises((OSError, subprocess.CalledProcessError)):
        tbbuild.build_bind()


def test_rebuilds_for_another_torch(elsewhere, monkeypatch):
    monkeypatch.setenv("CXX", compiler(elsewhere, "cxx", "anew"))
    (elsewhere / "bind.so").write_bytes(b"torch 0.1, python 3.12\0")  # newer than its sources
    tbbuild.build()
    assert (elsewhere / "bind.so").read_text() == "anew"


def test_what_is_built_is_kept():
    tbbuild.build()
    before = os.stat(tbbuild.BIND).st_mtime_ns
    tbbuild.build()
    assert os.stat(tbbuild.BIND).st_mtime_ns == before
