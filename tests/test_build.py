"""The library's build where the binding's native argument checks cannot be
built: libdg.so needs hipcc alone."""
import os
import sys

import pytest

from moe_grouped_gemm_scaled_amd import build


def no_torch():
    raise ImportError("No module named 'torch'")


@pytest.mark.parametrize("command", [lambda: [sys.executable, "-c", "raise SystemExit('no header')"],
                                     lambda: ["/nonexistent/g++"], no_torch],
                         ids=["compiler fails", "no compiler", "no torch"])
def test_library_without_the_native_checks(tmp_path, monkeypatch, capsys, command):
    monkeypatch.setattr(build, "SOURCES", ["layer_api.cpp"])          # enough of a library to link
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libdg.so"))
    monkeypatch.setattr(build, "ARGS", str(tmp_path / "_args.so"))
    monkeypatch.setattr(build, "_args_command", command)
    (tmp_path / "_args.so").write_bytes(b"older")
    assert build.build() == build.LIB and os.path.getsize(build.LIB) > 0
    assert not os.path.exists(build.ARGS)                             # checks of an older source do not stay
    assert "_args.so was not built" in capsys.readouterr().err
